"""u and du of the adapters' bf16 products at the ends of binary32: beyond bf16's largest
value, and infinite."""
import math

import pytest
import torch

import mixture_experts_layer_06_amd as moe
from test_gpu_ffn import DT, check, half_step

pytestmark = pytest.mark.gpu

LAST = 2.0 ** 128 - 2.0 ** 120  # the largest bf16 value
NEXT = 2.0 ** 120 - 2.0 ** 112  # LAST + NEXT is a binary32 value that rounds to infinity in bf16
ENDS = [(LAST, NEXT), (-LAST, -NEXT), (LAST, 0.0), (3.0e38, 0.0), (math.inf, 0.0), (-math.inf, 1.0), (1.0, 0.0)]


@pytest.mark.parametrize("R", [1, 4, 24])
@pytest.mark.parametrize("f", [1.0, 0.125])
@pytest.mark.parametrize("rest", [0.0, 1.0])
def test_values_at_the_end_of_binary32(R, f, rest):
    """u beyond what bf16 rounds to a finite value, and infinite: out is what the formula
    gives, infinite where it says so, and NaN only where it multiplies an infinity by 0
    (ranks whose factors are 0). Products with the scales are exact."""
    gen = torch.Generator().manual_seed(R)
    x = torch.tensor(ENDS).bfloat16()
    a = torch.full((1, 2, R), rest)
    a[0, :, 0] = 1.0
    b = (torch.rand((1, R, 40), generator=gen) * 2.0 ** -7 + 2.0 ** -8).bfloat16()
    off = torch.tensor([0, len(ENDS)], dtype=torch.int32).cuda()
    out = moe.lora(x.cuda(), a.bfloat16().cuda(), b.cuda(), off, scale=torch.tensor([f]).cuda()).cpu().double()
    u = (x.double()[:, :, None] * a.bfloat16().double()).sum(1)
    want = f * (u[:, :, None] * b.double()).sum(1)
    ok = torch.isfinite(want)
    assert ok.any() and torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out[torch.isinf(want)], want[torch.isinf(want)])
    # 16 bits of u, 2 R sums of its terms of one sign, the result's rounding
    rel = half_step(torch.bfloat16) + 2.0 ** -15 + 2 * R * 2.0 ** -23
    assert ((out - want).abs()[ok] <= rel * want.abs()[ok]).all()


@pytest.mark.parametrize("dw", ["bf16", "f32"])
def test_large_u_in_the_gradient(dw):
    """u (binary32 from the caller) between bf16's and binary32's largest values."""
    u = torch.tensor([[3.4e38, -3.4028234e38, 1.0, 3.3962e38, -3.39e38]])
    R, H, N = u.shape[1], 8, 24
    dout = (torch.rand((1, N), generator=torch.Generator().manual_seed(1)) + 0.5).bfloat16() * 2.0 ** -6
    x, a, b = torch.ones((1, H)).bfloat16(), torch.zeros((1, H, R)).bfloat16(), torch.zeros((1, R, N)).bfloat16()
    off = torch.tensor([0, 1], dtype=torch.int32).cuda()
    _, _, db = moe.lora_bwd(dout.cuda(), x.cuda(), u.cuda(), a.cuda(), b.cuda(), off, dw_dtype=DT[dw])
    want = u[0].double()[:, None] * dout.double()
    bound = (half_step(DT[dw]) + 2.0 ** -22 + (2.0 ** -15 if dw == "bf16" else 0.0)) * want.abs()
    check(db[0], want, bound, "db")
    assert torch.isfinite(db.float()).all()
