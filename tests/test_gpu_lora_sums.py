"""fp32 gradients of bf16 rows keep all 24 bits of u and du."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe
from test_gpu_ffn import STEP, check
from test_gpu_lora import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [1, 5, 16, 20, 33, 64, 100, 128])
def test_every_bit_of_u_and_du(R):
    """One row to an adapter and factors of one: db is u and da is du, bit for bit. du is
    one product of scale and b, rounded once."""
    e, H, N = 5, 72, 1
    gen = torch.Generator().manual_seed(R)
    x, dout = torch.ones((e, H)).bfloat16(), torch.ones((e, N)).bfloat16()
    a, b = torch.randn((e, H, R), generator=gen).bfloat16(), torch.randn((e, R, N), generator=gen).bfloat16()
    scale, u = torch.rand((e,), generator=gen) + 0.5, torch.randn((e, R), generator=gen)
    off = torch.arange(e + 1, dtype=torch.int32).cuda()
    _, da, db = moe.lora_bwd(dout.cuda(), x.cuda(), u.cuda(), a.cuda(), b.cuda(), off, scale=scale.cuda(),
                             dw_dtype=torch.float32)
    du = scale[:, None] * b[:, :, 0].float()
    assert torch.equal(da.cpu(), du[:, None, :].expand(e, H, R))
    _, _, db1 = moe.lora_bwd(dout.cuda(), x.cuda(), u.cuda(), a.cuda(), b.cuda(), off, dw_dtype=torch.float32)
    assert torch.equal(db1.cpu(), u[:, :, None])
    assert torch.equal(db.cpu(), (scale[:, None] * u)[:, :, None])


@pytest.mark.parametrize("counts,H,N,R", [([3, 0, 9], 136, 264, 16), ([300, 41], 257, 401, 20), ([700, 30], 512, 640, 64),
                                          ([2600, 9], 96, 128, 128), ([150], 1024, 1024, 8)])
def test_fp32_gradients_of_bf16_rows(counts, H, N, R):
    """Sums of exact products in binary32: nothing is left out of u or du. n additions of
    three terms' products are off by n steps of their magnitudes, du by N + 4."""
    c = Case(counts, H, N, R, "bf16", H + R, idle=3, extra=2)
    dout, x, u, a, b, scale = c.dev("dout", "x", "u", "a", "b", "scale")
    _, da, db = moe.lora_bwd(dout, x, u, a, b, c.offsets, rows=c.rows_d, scale=scale, need_dx=False,
                             dw_dtype=torch.float32)
    for e, s, t, f in c.segs():
        d, xr, b64, v = c.dout[t].double(), c.x[t].double(), c.b[e].double(), c.u[s].double()
        du, w = f * (d @ b64.T), abs(f) * (d.abs() @ b64.abs().T)
        edu = (N + 4) * STEP * w + STEP * du.abs()
        n = 3 * len(t) + 40
        g = xr.T @ du
        check(da[e], g, xr.abs().T @ edu + n * STEP * (xr.abs().T @ du.abs()) + 2.0 ** -24 * g.abs(), f"da of {e}")
        g = f * (v.T @ d)
        check(db[e], g, abs(f) * n * STEP * (v.abs().T @ d.abs()) + 2.0 ** -24 * g.abs(), f"db of {e}")


def test_sums_lose_no_bits_on_average():
    """The norm of the error, which two terms of 8 bits would leave at 2^-18 of each
    product and binary32 sums of 40 rows leave at a few 2^-24."""
    c = Case([40, 33], 256, 320, 16, "bf16", 5)
    dout, x, u, a, b, scale = c.dev("dout", "x", "u", "a", "b", "scale")
    db = moe.lora_bwd(dout, x, u, a, b, c.offsets, rows=c.rows_d, scale=scale, need_dx=False, need_da=False,
                      dw_dtype=torch.float32)[2]
    for e, s, t, f in c.segs():
        g = f * (c.u[s].double().T @ c.dout[t].double())
        # 2^-24 sqrt(40) from the sums at most, against 2^-18 / sqrt(3) from dropped bits
        assert (db[e].cpu().double() - g).norm() <= 2.0 ** -21 * g.norm()
