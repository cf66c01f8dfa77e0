"""Gates at the ends of their types: the activations and their derivatives neither
overflow nor lose their limits. Inputs are exact, so that act(g) is off by the
activation's own error only: relative (|g| + g^2 + 8) * 2^-23 (the exponential's
argument is rounded; g^2 for GELU only) plus one rounding to the type; below the
smallest normal number 2^-126 hardware exponentials and reciprocals return 0,
which 2^-126 * |g| covers where that factor is multiplied with g."""
import math

import pytest
import torch

import mixture_experts_layer_06_amd as moe

pytestmark = pytest.mark.gpu

ACTS = {"silu": moe.ACT_SILU, "gelu": moe.ACT_GELU, "relu": moe.ACT_RELU, "none": moe.ACT_NONE}
GATES = [0.0, -0.0, 2.0 ** -126, -2.0 ** -126, 2.0 ** -60, -1.2734375, 0.7, -0.7, 5.0, -5.0, 13.0, -13.0, 60.0, -60.0, 87.0,
         -87.0, 89.0, -89.0, 104.0, -104.0, 1e4, -1e4, 1e19, -1e19, 3e38, -3e38]


def act64(g, name):
    """act(g), act'(g) and the sum of its terms' magnitudes."""
    if name == "silu":
        s, r = torch.sigmoid(g), torch.sigmoid(-g)
        return g * s, s * (1 + g * r), s * (1 + g.abs() * r)
    if name == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        q = g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        return g * p, p + q, p + q.abs()
    if name == "relu":
        return torch.relu(g), (g > 0).double(), (g > 0).double()
    return g, torch.ones_like(g), torch.ones_like(g)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("width", [32, 27])  # vectors of the pointwise pass, and single elements
def test_extreme_gates(act, dt, width):
    g = torch.tensor((GATES + [0.0] * width)[:width]).to(dt)
    keep = g.double().abs()
    half = torch.finfo(dt).eps / 2
    rel = (keep + (keep * keep if act == "gelu" else 0) + 8) * 2.0 ** -23
    rel = rel.clamp(max=1.0)  # where the factor vanishes altogether
    eye = torch.eye(width).to(dt)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    a, p, terms = act64(g.double(), act)
    # forward: x = 1, Wg = g, Wu = 1: one product each, exact
    one = torch.ones((1, 1), dtype=dt, device="cuda")
    out, gate, up = moe.gmm_glu(one, g.cuda().reshape(1, 1, -1), torch.ones((1, 1, width), dtype=dt, device="cuda"),
                                off, act=ACTS[act], save=True)
    flushed = 2.0 ** -126 * (1 + keep)
    got = out[0].cpu().double()
    assert torch.equal(gate[0].cpu().abs(), torch.where(g.abs() < 2.0 ** -126, g * 0, g).abs()) and bool((up == 1).all())
    assert torch.isfinite(got).all()
    assert bool(((got - a).abs() <= (rel + half + rel * half) * a.abs() + flushed).all()), (got - a)
    # backward: d = u = 1, Wg = I, Wu = 0, so da is dg; and x = 1, so dw_gate = dg, dw_up = du
    n = torch.ones((1, width), dtype=dt, device="cuda")
    zero = torch.zeros((1, width, width), dtype=dt, device="cuda")
    da, dwg, dwu = moe.gmm_glu_bwd(n, g.cuda().reshape(1, -1), n, n, eye.cuda().reshape(1, width, width), zero, off,
                                   act=ACTS[act])
    for got, want, size in ((da[0], p, terms), (dwg[0, 0], p, terms), (dwu[0, 0], a, a.abs())):
        got = got.cpu().double()
        assert torch.isfinite(got).all()
        assert bool(((got - want).abs() <= (rel + 2 * half + 2 * rel * half) * size + flushed).all()), (got - want)
