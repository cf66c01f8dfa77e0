"""Calls that take a workspace give the same bits whatever it held before: every byte
0xFF (NaN as a number, -1 as a count) or zero."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe
from test_gpu_ffn import DT
from test_gpu_lora import Case

pytestmark = pytest.mark.gpu


def scratch(n, fill):
    return torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")


def same(call, size):
    """call(ws) with both fillings: the results' bits, and none of them NaN."""
    for a, b in zip(call(scratch(size, 0xFF)), call(scratch(size, 0))):
        if a is not None:
            assert not torch.isnan(a.float()).any() and torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 20, 33, 36, 100, 127])
def test_adapters(R, dt):
    c = Case([40, 0, 33, 7], 264, 520, R, dt, R, idle=3, extra=2)
    size = moe.lora_workspace_size(moe.BF16 if dt == "bf16" else moe.F32, c.e, c.M, c.H, c.N, R)
    base = c.base.cuda()
    same(lambda ws: (c.forward(base=base, ws=ws),), size)
    dout, x, u, a, b, scale, dx = c.dev("dout", "x", "u", "a", "b", "scale", "dx")
    size = moe.lora_bwd_workspace_size(moe.BF16 if dt == "bf16" else moe.F32, c.e, c.M, c.H, c.N, R)
    same(lambda ws: moe.lora_bwd(dout, x, u, a, b, c.offsets, rows=c.rows_d, scale=scale, base=dx, ws=ws), size)


@pytest.mark.parametrize("counts,H,N,R,dt", [
    # partial sums added by a launch of their own
    ([9000, 0, 7000], 1536, 72, 100, "bf16"), ([12000, 9598], 1536, 72, 49, "f32"), ([16000, 5], 1540, 64, 52, "bf16"),
    # rows split for the weight gradients, large tiles
    ([2600, 0, 500, 1], 520, 1032, 4, "bf16"), ([2600, 40], 257, 401, 3, "f32"), ([4000], 130, 1031, 12, "bf16"),
])
def test_adapters_of_many_rows(counts, H, N, R, dt):
    c = Case(counts, H, N, R, dt, H, idle=2)
    code = moe.BF16 if dt == "bf16" else moe.F32
    base = c.base.cuda()
    same(lambda ws: c.forward(base=base, u=True, ws=ws)[:1], moe.lora_workspace_size(code, c.e, c.M, H, N, R))
    dout, x, u, a, b, scale, dx = c.dev("dout", "x", "u", "a", "b", "scale", "dx")
    for dw in {dt, "f32"}:
        same(lambda ws: moe.lora_bwd(dout, x, u, a, b, c.offsets, rows=c.rows_d, scale=scale, base=dx, ws=ws,
                                     dw_dtype=DT[dw]), moe.lora_bwd_workspace_size(code, c.e, c.M, H, N, R))


@pytest.mark.parametrize("T,E,K", [(5000, 8, 2), (20011, 61, 4), (65536, 256, 8)])
def test_router_loss(T, E, K):
    gen = torch.Generator().manual_seed(T)
    scores = torch.randn((T, E), generator=gen).cuda()
    idx = scores.topk(K, 1).indices.to(torch.int32)
    size = moe.router_loss_workspace_size(T, E, K)
    assert size > 0
    same(lambda ws: tuple(moe.router_loss(scores, idx, ws=ws).values()), size)


@pytest.mark.parametrize("T,N,kind", [(3, 7, "layer"), (700, 1501, "layer"), (1, 4096, "rms"), (300, 9000, "layer"),
                                      (600, 20000, "rms"), (4100, 256, "layer")])
def test_norm_gradients(T, N, kind):
    gen = torch.Generator().manual_seed(T + N)
    d, z, r = (torch.randn((T, N), generator=gen).cuda() for _ in range(3))
    w, g, b = (torch.randn(N, generator=gen).cuda() for _ in range(3))
    layer = kind == "layer"
    how = dict(w_post=w, b_post=b if layer else None, gate=g, w_pre=w, kind=moe.NORM_LAYER if layer else moe.NORM_RMS)
    same(lambda ws: tuple(moe.block_norm_bwd(d, r, z, r, ws=ws, **how).values()),
         moe.block_norm_bwd_workspace_size(T, N))
