"""Rounding of long sums in the gated feed-forward and the grouped GEMM's gradients:
normwise against fp64, ||got - want|| / ||want|| on normal operands, where one
running binary32 sum over the whole reduction would exceed the limit.

Limits. An MFMA adds the products of one step (4 k values in binary32, 32 in
bf16) to its accumulator and is off by up to one step 2^-23 of the sum at hand;
taken as spread evenly, rms 2^-23 / sqrt(3) = 6.9e-8. After m steps on normal
products the sum has grown with sqrt(m), and these errors add up to
sqrt(m / 2) * 6.9e-8 of it. An addition to a total is correctly rounded, rms
2^-24 / sqrt(3) = 3.4e-8, and t of them add up to sqrt(t / 2) * 3.4e-8 likewise.
Sums with totals, over n values, in pieces of p:
    limit(n, p, step) = 1.1 * hypot(sqrt(p / step / 2) * 6.9e-8, sqrt(n / p / 2) * 3.4e-8)
(1.1: the norms are those of finite samples). p is 128 in binary32. fp32 results
of bf16 operands have p = 4096; a single sum over 65536 products was off by
1.6e-6, over 262144 by 3.3e-6, a binary32 one over 16384 by 2.3e-6."""
import math

import pytest
import torch

import mixture_experts_layer_06_amd as moe

pytestmark = pytest.mark.gpu


def limit(n, piece, step):
    return 1.1 * math.hypot(math.sqrt(piece / step / 2) * 2 ** -23 / math.sqrt(3),
                            math.sqrt(n / piece / 2) * 2 ** -24 / math.sqrt(3))


def normwise(got, want):
    assert torch.isfinite(got).all()
    return float((got.double() - want).norm() / want.norm())


def uneven(experts, long, short, dt, Hin, N, gather, seed=0):
    """Rows of `experts` experts of `short` rows each but for the second, which has
    `long` (the first of one expert): x rows, output gradients, offsets, gather
    indexes and the long expert's rows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    which = min(1, experts - 1)
    counts = [short] * experts
    counts[which] = long
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    A = sum(counts)
    lo = sum(counts[:which])
    d = torch.randn((A, N), generator=gen, device="cuda").to(dt)
    x = torch.randn((A, Hin), generator=gen, device="cuda").to(dt)
    rows = torch.randperm(A, generator=gen, device="cuda").to(torch.int32) if gather else None
    xr = x if rows is None else x[rows.long()]
    return x, d, offsets, rows, which, slice(lo, lo + long), xr


def check_uneven(experts, long, short, dt, Hin, N, gather, piece, step):
    x, d, offsets, rows, which, s, xr = uneven(experts, long, short, dt, Hin, N, gather)
    dw = moe.gmm_wgrad(x, d, offsets, rows=rows, out_dtype=torch.float32)
    err = normwise(dw[which], xr[s].double().T @ d[s].double())
    assert err <= limit(long, piece, step), f"long expert: {err:.2e}"
    if which:  # and a short one beside it
        err = normwise(dw[0], xr[:short].double().T @ d[:short].double())
        assert err <= limit(max(short, piece), min(short, piece) + step, step), f"short expert: {err:.2e}"


# The average load is a few hundred rows, one expert has 16421.
@pytest.mark.parametrize("experts,Hin,N,gather", [
    (64, 333, 333, True), (64, 333, 333, False),   # rows of any alignment
    (256, 1300, 3, False),                         # fewer than four columns
    (64, 512, 512, True), (8, 260, 264, False),    # rows on 16 bytes
    (1, 99, 54, False), (1, 516, 520, True),       # rows split over blocks
])
def test_fp32_weight_gradients_of_one_long_expert(experts, Hin, N, gather):
    check_uneven(experts, 16421, 8, torch.float32, Hin, N, gather, 128, 4)


# fp32 results of bf16 operands: large and small DMA tiles, rows split over
# blocks, rows of any alignment, fewer than four columns.
@pytest.mark.parametrize("experts,Hin,N,gather", [
    (64, 512, 512, True), (64, 512, 512, False),
    (64, 128, 128, True), (64, 128, 136, False),
    (1, 4096, 2048, False),
    (1, 256, 256, True), (1, 136, 72, False),
    (64, 333, 333, True), (64, 333, 332, False), (256, 1300, 3, False),
    (2, 99, 54, True),
])
def test_fp32_weight_gradients_of_bf16_rows(experts, Hin, N, gather):
    # 16 parts of one expert's rows are still 16 times a piece
    check_uneven(experts, 65536 + 37 if experts > 1 else 262144 + 37, 8, torch.bfloat16, Hin, N, gather, 4096, 32)


# Reductions of 4224 k values: DMA tiles of 64 x 128 and 128 x 128, register-staged
# tiles of any alignment, large (128 x 128) and small.
@pytest.mark.parametrize("counts,Hin,N", [
    ([300, 0, 700, 40], 4224, 1024), ([2304], 4224, 2048), ([700, 1300], 4225, 1501), ([5, 0, 130], 4226, 75),
    ([9], 4224, 64),
])
def test_fp32_projections_of_long_rows(counts, Hin, N):
    gen = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    A, e = sum(counts), len(counts)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    x, wg, wu = mk(A, Hin), mk(e, Hin, N), mk(e, Hin, N)
    _, gate, up = moe.gmm_glu(x, wg, wu, offsets, act=moe.ACT_NONE, save=True)
    lo = 0
    for i, n in enumerate(counts):
        for got, w in ((gate, wg), (up, wu)):
            if n:
                err = normwise(got[lo:lo + n], x[lo:lo + n].double() @ w[i].double())
                assert err <= limit(Hin, 128, 4), f"expert {i}: {err:.2e}"
        lo += n


@pytest.mark.parametrize("counts,Hin,N", [
    ([300, 0, 700, 40], 1024, 4224), ([2304], 2048, 4224), ([700, 1300], 1501, 4225), ([5, 0, 130], 75, 4226),
])
def test_fp32_row_gradients_of_long_rows(counts, Hin, N):
    gen = torch.Generator(device="cuda").manual_seed(2)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    A, e = sum(counts), len(counts)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    d, w, w2 = mk(A, N), mk(e, Hin, N), mk(e, Hin, N)
    one, none = torch.ones_like(d), moe.ACT_NONE
    da = moe.gmm_dgrad(d, w, offsets)
    # act'(g) = 1 and g = u = 1: both projections' gradients are d
    both, _, _ = moe.gmm_glu_bwd(d, one, one, mk(A, Hin), w, w2, offsets, act=none, need_dw=False)
    lo = 0
    for i, n in enumerate(counts):
        if n:
            s = slice(lo, lo + n)
            err = normwise(da[s], d[s].double() @ w[i].double().T)
            assert err <= limit(N, 128, 4), f"expert {i}: {err:.2e}"
            err = normwise(both[s], d[s].double() @ (w[i].double() + w2[i].double()).T)
            assert err <= limit(2 * N, 128, 4), f"expert {i}, both projections: {err:.2e}"
        lo += n


# Large tiles whose waves have no columns (56 of 256 left) or no rows (104 of 256).
@pytest.mark.parametrize("Hin,N,gather", [(872, 3896, False), (872, 3896, True), (1024, 3896, False), (872, 4096, False)])
def test_fp32_weight_gradients_of_partial_tiles(Hin, N, gather):
    check_uneven(4, 65536 + 37, 8, torch.bfloat16, Hin, N, gather, 4096, 32)


@pytest.mark.parametrize("extra", [4, 1])
@pytest.mark.parametrize("counts,Hin,N", [([9001], 136, 72), ([4100, 0, 2999], 264, 40), ([300, 5, 0, 700], 520, 264)])
def test_weight_gradients_of_rows_off_16_bytes(counts, Hin, N, extra):
    """Dense N on 16 bytes, but gradients in a tensor whose rows are not: another
    kernel, with the workspace of the size query, which does not know the stride.
    Integer operands, whose sums are exact: the same bits as dense."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    A, e = sum(counts), len(counts)
    small = lambda m, *s: torch.randint(-m, m + 1, s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    x, d, g, u, w = small(2, A, Hin), small(1, A, N), small(1, A, N), small(1, A, N), small(1, e, Hin, N)
    _, dwg, dwu = moe.gmm_glu_bwd(d, g, u, x, w, w, offsets, act=moe.ACT_NONE, need_da=False)
    wide = torch.full((e, Hin, 2 * N + extra), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.gmm_glu_bwd_workspace_size(moe.BF16, e, A, Hin, N), dtype=torch.uint8, device="cuda")
    moe.gmm_glu_bwd(d, g, u, x, w, w, offsets, act=moe.ACT_NONE, need_da=False, dw_gate=wide[:, :, :N],
                    dw_up=wide[:, :, N:2 * N], ws=ws)
    assert torch.equal(wide[:, :, :N], dwg) and torch.equal(wide[:, :, N:2 * N], dwu)
    assert bool((wide[:, :, 2 * N:] == 7.0).all())
    lo = 0
    for i, n in enumerate(counts):
        want = x[lo:lo + n].double().T @ (d[lo:lo + n].double() * u[lo:lo + n].double())
        assert torch.equal(dwg[i], want.to(torch.bfloat16))
        lo += n


@pytest.mark.parametrize("experts,Hin,N,dt", [(64, 512, 512, torch.bfloat16), (64, 333, 333, torch.bfloat16),
                                              (1, 256, 256, torch.bfloat16), (64, 333, 333, torch.float32)])
def test_graph_replays_of_sums_in_pieces(experts, Hin, N, dt):
    """Pieces are added to what this launch stored, whatever the output held before."""
    x, d, offsets, rows, *_ = uneven(experts, 16421, 8, dt, Hin, N, True)
    out = torch.full((experts, Hin, N), float("nan"), device="cuda")
    n = moe.gmm_wgrad_workspace_size(moe.F32 if dt == torch.float32 else moe.BF16, experts, x.shape[0], Hin, N)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    want = moe.gmm_wgrad(x, d, offsets, rows=rows, out=out, ws=ws).clone()
    assert torch.isfinite(want).all()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.gmm_wgrad(x, d, offsets, rows=rows, out=out, ws=ws)
    x0 = x.clone()
    for k in range(4):
        x.copy_(x0 if k % 2 == 0 else -x0)
        out.fill_(float("inf"))
        graph.replay()
        torch.cuda.synchronize()
        assert k % 2 or torch.equal(out, want)  # (a bf16 MFMA of negated operands rounds otherwise)
        assert torch.equal(out, moe.gmm_wgrad(x, d, offsets, rows=rows, out_dtype=torch.float32))
