"""Tokens without a part in the losses get no part of their gradient, whatever its size."""
import math

import pytest
import torch

import mixture_experts_layer_06_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,K", [(2, 1), (8, 2), (61, 4), (128, 8), (200, 3)])
@pytest.mark.parametrize("dloss", [(math.inf, 0.0), (0.0, -math.inf), (math.nan, 1.0), (3e38, 3e38)])
def test_gradients_beyond_the_numbers(E, K, dloss):
    """A loss scale that overflowed: rows that are masked, or whose scores are all -inf,
    keep 0 from the losses and the gates' part alone."""
    T = 300
    gen = torch.Generator().manual_seed(E)
    scores = torch.randn((T, E), generator=gen)
    idx = scores.topk(K, 1).indices.to(torch.int32).cuda()
    scores[::7] = -math.inf
    scores = scores.cuda()
    mask = (torch.rand((T,), generator=gen) < 0.6).cuda()
    dead = ~mask | torch.isinf(scores).all(1)
    r = moe.router_loss(scores, idx, mask=mask)
    assert r["tokens"].item() == int((~dead).sum())
    dl = torch.tensor(dloss, device="cuda")
    got = moe.router_loss_bwd(scores, idx, r["counts"], r["tokens"], dloss=dl, mask=mask)
    assert (got[dead] == 0).all()
    gate = torch.softmax(torch.randn((T, K), generator=gen), 1).cuda()
    dgate = torch.randn((T, K), generator=gen).cuda()
    got = moe.router_loss_bwd(scores, idx, r["counts"], r["tokens"], dloss=dl, gate=gate, dgate=dgate, mask=mask)
    alone = moe.router_loss_bwd(scores, idx, gate=gate, dgate=dgate)
    assert torch.equal(got[dead], alone[dead])
