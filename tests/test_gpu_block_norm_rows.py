"""More rows than one launch may have threads for (2^32 of them)."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe

pytestmark = pytest.mark.gpu


def test_rows_of_two_launches():
    """8.5 million rows of 2056, 512 threads to a row; the rows around the launches' border,
    the first and the last get what they get alone, with their own gates."""
    T, N = 2 ** 23 + 100000, 2056
    z = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    block = torch.randn((4096, N), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    for i in range(0, T, 4096):
        z[i:i + 4096] = block[:min(4096, T - i)]
    gate = torch.rand((T, 1), device="cuda") + 0.5
    w = torch.rand(N, device="cuda") + 0.5
    r, h = torch.full_like(z, 7.0), torch.full_like(z, 7.0)
    moe.block_norm(z, None, w, gate=gate, w_pre=w, r_out=r, h=h)
    for lo in (0, 2 ** 23 - 600, 2 ** 23 - 8, T - 300):
        n = min(1200, T - lo)
        rows = torch.arange(lo, lo + n, device="cuda") % 4096
        ro, one = moe.block_norm(block[rows], None, w, gate=gate[lo:lo + n].clone(), w_pre=w)
        assert torch.equal(r[lo:lo + n], ro) and torch.equal(h[lo:lo + n], one)
    del z, r, h
    torch.cuda.empty_cache()
