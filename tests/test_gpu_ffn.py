"""The gated expert feed-forward and the grouped GEMM's gradients against plain
fp64 computations of the same operands (CPU, torch double).

Tolerances, element by element. A bf16 result is off by at most half a step,
2^-8 of its value; an fp32 one by 2^-24. A sum of n exact products carried in
binary32 is off by at most n * 2^-23 * sum|products| (one rounding of at most
one step per addition). The activation is off by (|g| + 8) * 2^-23 relative: the
exponential's argument g * log2(e) is rounded, which moves e^g by |g| steps, and
a few more steps come from the exponential, the reciprocal and the products;
the terms of its derivative likewise. GELU's exponent is g^2/2, whose rounding
(one step of its own value, in the square and again in the product with
log2(e)) moves the exponential by g^2/2 steps each: (|g| + g^2 + 8) * 2^-23. The bounds of the backward pass propagate
these through its formulas, with dg and du rounded to the tensors' type."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_06_amd as moe

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = 2.0 ** -23
ACTS = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}


def half_step(dt):
    return 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24


def act64(g, name):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return 0.5 * g * torch.erfc(-g / math.sqrt(2.0))
    return torch.relu(g) if name == "relu" else g


def dact64(g, name):
    """act'(g) and the sum of its terms' magnitudes."""
    if name == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * torch.sigmoid(-g)), s * (1 + g.abs() * torch.sigmoid(-g))
    if name == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        q = g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        return p + q, p + q.abs()
    if name == "relu":
        d = (g > 0).double()
        return d, d
    return torch.ones_like(g), torch.ones_like(g)


def act_rel(g, name):
    """Relative error of act(g) and of act'(g)'s terms."""
    return (g.abs() + (g * g if name == "gelu" else 0) + 8) * STEP


class Case:
    """Operands on the GPU and their fp64 copies; rows grouped by expert."""

    def __init__(self, counts, Hin, N, dt, seed, gather=True, fused=False, tail=0, T=None):
        gen = torch.Generator().manual_seed(seed)
        self.dt = DT[dt]
        self.counts, self.Hin, self.N = list(counts), Hin, N
        self.e = len(counts)
        self.A = sum(counts) + tail  # tail: rows behind the last expert's
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.off = off
        self.offsets = torch.from_numpy(off).cuda()
        self.div = 3
        T = T or max(1, (self.A + 2) // 3)

        def make(*shape, scale=1.0):
            return (torch.randn(shape, generator=gen) * scale).to(self.dt)

        if gather:
            rows = torch.randint(0, T * self.div, (self.A,), generator=gen, dtype=torch.int32)
            self.rows = rows.cuda()
            self.x = make(T, Hin)
            self.xr = self.x[(rows // self.div).long()].double()
        else:
            self.rows = None
            self.x = make(self.A, Hin)
            self.xr = self.x.double()
        if fused:
            w = make(self.e, Hin, 2 * N, scale=Hin ** -0.5)
            wd = w.cuda()
            self.wg, self.wu = wd[:, :, :N], wd[:, :, N:]
            self.wg64, self.wu64 = w[:, :, :N].double(), w[:, :, N:].double()
        else:
            wg, wu = make(self.e, Hin, N, scale=Hin ** -0.5), make(self.e, Hin, N, scale=Hin ** -0.5)
            self.wg, self.wu = wg.cuda(), wu.cuda()
            self.wg64, self.wu64 = wg.double(), wu.double()
        self.gate, self.up, self.dout = make(self.A, N, scale=2.0), make(self.A, N), make(self.A, N)
        self.x = self.x.cuda()

    def segs(self):
        return [(e, slice(int(a), int(b))) for e, (a, b) in enumerate(zip(self.off, self.off[1:])) if b > a]


def check(got, want, bound, what):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} elements off by up to {worst:.3e} beyond the bound"


def check_glu(c, act, **kw):
    fill = 7.0
    out, gate, up = (torch.full((c.A, c.N), fill, dtype=c.dt, device="cuda") for _ in range(3))
    moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, act=ACTS[act], rows=c.rows, row_div=c.div, out=out, gate=gate, up=up, **kw)
    bare = moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, act=ACTS[act], rows=c.rows, row_div=c.div, **kw)
    torch.cuda.synchronize()
    h = half_step(c.dt)
    covered = int(c.off[-1])
    assert torch.equal(bare[:covered], out[:covered])  # saving the projections changes nothing
    for t in (out, gate, up):
        assert bool((t[covered:] == fill).all())  # rows no expert covers stay as they were
    for e, s in c.segs():
        x = c.xr[s]
        g, u = x @ c.wg64[e], x @ c.wu64[e]
        n = c.Hin * STEP
        eg, eu = n * (x.abs() @ c.wg64[e].abs()), n * (x.abs() @ c.wu64[e].abs())
        check(gate[s], g, eg + h * g.abs() + h * eg, f"gate of expert {e}")
        check(up[s], u, eu + h * u.abs() + h * eu, f"up of expert {e}")
        a = act64(g, act)
        ea = 1.13 * eg + act_rel(g, act) * a.abs()  # |act'| < 1.13
        want = a * u
        b = ea * u.abs() + a.abs() * eu + ea * eu
        check(out[s], want, b + h * (want.abs() + b), f"out of expert {e}")


def check_bwd(c, act, **kw):
    fill = 7.0
    da = torch.full((c.A, c.Hin), fill, dtype=c.dt, device="cuda")
    args = [t.cuda() for t in (c.dout, c.gate, c.up)]
    da, dwg, dwu = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, act=ACTS[act], rows=c.rows, row_div=c.div, da=da, **kw)
    torch.cuda.synchronize()
    h = half_step(c.dt)
    assert bool((da[int(c.off[-1]):] == fill).all())
    zero = torch.zeros((c.Hin, c.N), dtype=torch.float64)
    for e in range(c.e):
        s = slice(int(c.off[e]), int(c.off[e + 1]))
        rows = s.stop - s.start
        if rows == 0:
            check(dwg[e], zero, zero, f"dw_gate of empty expert {e}")
            check(dwu[e], zero, zero, f"dw_up of empty expert {e}")
            continue
        d, g, u, x = c.dout[s].double(), c.gate[s].double(), c.up[s].double(), c.xr[s]
        a = act64(g, act)
        p, pm = dact64(g, act)
        dg, du = d * u * p, d * a
        rel = act_rel(g, act)
        eg = (d * u).abs() * pm * rel
        eu = (d * a).abs() * rel
        eg, eu = eg + h * (dg.abs() + eg), eu + h * (du.abs() + eu)
        for got, dd, ed, what in ((dwg, dg, eg, "dw_gate"), (dwu, du, eu, "dw_up")):
            want = x.T @ dd
            b = x.abs().T @ ed + rows * STEP * (x.abs().T @ (dd.abs() + ed))
            check(got[e], want, b + h * (want.abs() + b), f"{what} of expert {e}")
        want = dg @ c.wg64[e].T + du @ c.wu64[e].T
        wga, wua = c.wg64[e].abs().T, c.wu64[e].abs().T
        b = eg @ wga + eu @ wua + 2 * c.N * STEP * ((dg.abs() + eg) @ wga + (du.abs() + eu) @ wua)
        check(da[s], want, b + h * (want.abs() + b), f"da of expert {e}")


# counts, Hin, N, dtype, gather, fused, rows behind the last expert
GLU_CASES = {
    "one_row": ([1], 64, 64, "bf16", True, False, 0),
    "one_row_f32": ([1], 1, 1, "f32", True, False, 0),
    "one_row_odd": ([0, 1, 0], 37, 19, "bf16", False, False, 1),
    "decode": ([0, 1, 3, 0, 2, 16, 1, 0], 512, 192, "bf16", True, False, 0),
    "decode_wide": ([1, 0, 0, 2], 4096, 96, "bf16", True, False, 2),
    "decode_k_tail": ([2, 5, 0, 17], 1000, 264, "bf16", True, True, 0),
    "decode_33": ([33, 1, 47], 264, 320, "bf16", False, True, 3),
    "odd": ([5, 0, 130, 61, 1], 100, 75, "bf16", True, False, 4),
    "three_columns": ([5, 0, 33], 3, 130, "bf16", True, False, 0),
    "three_rows_f32": ([5, 0, 33], 130, 2, "f32", True, False, 1),
    "five_by_seven": ([5, 0, 33], 5, 7, "bf16", False, False, 1),
    "odd_aligned4": ([70, 3], 36, 44, "bf16", False, False, 0),
    # enough 128 x 128 tiles for every CU
    "odd_many": ([7 * i % 45 for i in range(48)], 515, 261, "bf16", True, False, 2),
    "aligned4_many": ([11 * i % 52 for i in range(48)], 516, 260, "bf16", False, False, 1),
    "f32_many": ([7 * i % 45 for i in range(48)], 516, 268, "f32", True, False, 2),
    "f32_long": ([400, 1700], 1100, 1104, "f32", True, False, 0),
    "f32_odd_many": ([5 * i % 33 for i in range(48)], 514, 259, "f32", False, False, 0),
    "f32": ([5, 0, 130, 61, 1], 100, 76, "f32", True, True, 4),
    # one expert with many 128 x 128 tiles (GLU, then dgrad); ragged experts on 64 x
    # 128 tiles; rows split for the weight gradients
    "f32_one_wide": ([2050], 260, 2052, "f32", True, True, 0),
    "f32_one_tall": ([2050], 4100, 136, "f32", False, False, 1),
    "f32_ragged": ([130, 0, 65, 1, 700, 64, 63, 300], 2580, 520, "f32", True, False, 3),
    "f32_split": ([6001], 516, 520, "f32", True, False, 0),
    "f32_odd": ([17, 129], 33, 35, "f32", False, False, 1),
    "tiles": ([256, 0, 300, 257], 128, 256, "bf16", True, False, 0),
    "tiles_fold": ([288, 289, 543, 16], 96, 136, "bf16", True, True, 5),
    "tiles_one_expert": ([700], 40, 520, "bf16", False, False, 0),
    "tiles_k_tail": ([513, 255], 1000, 24, "bf16", True, False, 0),
    "tiles_many": ([300, 1, 0, 90, 260, 33, 512, 64], 264, 392, "bf16", True, False, 7),
    # many rows over few weight tiles: the rows are split for the weight gradients
    "long_dense": ([9001], 136, 72, "bf16", False, False, 2),
    "long_gathered": ([4100, 0, 2999], 264, 40, "bf16", True, True, 0),
    "long_odd": ([4001, 3, 2050], 133, 71, "bf16", True, False, 1),
    "long_odd_f32": ([5003], 99, 54, "f32", False, False, 0),
    # more k slices than one block of a gather's row offsets
    "long_rows": ([1537, 511, 513], 2312, 520, "bf16", True, False, 1),
}


def case_of(name, **kw):
    counts, Hin, N, dt, gather, fused, tail = GLU_CASES[name]
    return Case(counts, Hin, N, dt, seed=sum(map(ord, name)), gather=gather, fused=fused, tail=tail, **kw)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("name", list(GLU_CASES))
def test_glu_parity(name, act):
    check_glu(case_of(name), act)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("name", list(GLU_CASES))
def test_glu_bwd_parity(name, act):
    check_bwd(case_of(name), act)


@pytest.mark.parametrize("name", list(GLU_CASES))
def test_gmm_gradients_parity(name):
    c = case_of(name)
    h = half_step(c.dt)
    dout, w = c.dout.cuda(), c.wg.contiguous()
    da = torch.full((c.A, c.Hin), 7.0, dtype=c.dt, device="cuda")
    moe.gmm_dgrad(dout, w, c.offsets, out=da)
    dw = moe.gmm_wgrad(c.x, dout, c.offsets, rows=c.rows, row_div=c.div)
    dw32 = moe.gmm_wgrad(c.x, dout, c.offsets, rows=c.rows, row_div=c.div, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert dw.dtype == c.dt and dw32.dtype == torch.float32
    assert bool((da[int(c.off[-1]):] == 7.0).all())
    for e in range(c.e):
        s = slice(int(c.off[e]), int(c.off[e + 1]))
        d, x = c.dout[s].double(), c.xr[s]
        want = d @ c.wg64[e].T
        b = c.N * STEP * (d.abs() @ c.wg64[e].abs().T)
        check(da[s], want, b + h * (want.abs() + b), f"da of expert {e}")
        want = x.T @ d
        b = (s.stop - s.start) * STEP * (x.abs().T @ d.abs())
        check(dw[e], want, b + h * (want.abs() + b), f"dw of expert {e}")
        check(dw32[e], want, b + 2.0 ** -24 * (want.abs() + b), f"fp32 dw of expert {e}")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_gradients_match_differences(act):
    """Directional derivatives of sum(out * dout) by central differences of the
    fp64 function, against the fp32 kernels' gradients."""
    c = Case([3, 0, 5], 12, 7, "f32", 5, gather=False)

    def loss(x, wg, wu):
        t = 0.0
        for e, s in c.segs():
            t += (act64(x[s] @ wg[e], act) * (x[s] @ wu[e]) * c.dout[s].double()).sum().item()
        return t

    out, gate, up = moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, act=ACTS[act], save=True)
    grads = moe.gmm_glu_bwd(c.dout.cuda(), gate, up, c.x, c.wg, c.wu, c.offsets, act=ACTS[act])
    at = [c.xr, c.wg64, c.wu64]
    gen = torch.Generator().manual_seed(1)
    step = 1e-4
    for i, grad in enumerate(grads):
        for _ in range(4):
            v = torch.randn(at[i].shape, generator=gen, dtype=torch.float64)
            lo, hi = list(at), list(at)
            lo[i], hi[i] = at[i] - step * v, at[i] + step * v
            want = (loss(*hi) - loss(*lo)) / (2 * step)
            terms = grad.cpu().double() * v
            # the difference quotient's error is O(step^2) = 1e-8 of third
            # derivatives of order one per term; each fp32 gradient element is
            # a sum of at most 2 N or 5 terms, off by below 64 * 2^-23
            tol = (64 * STEP + 1e-7) * terms.abs().sum().item() + 1e-6 * v.abs().sum().item()
            assert abs(terms.sum().item() - want) <= tol


def test_relu_gate_derivative_is_zero_at_zero():
    x = torch.ones((1, 8), device="cuda")
    w = torch.ones((1, 8, 8), device="cuda")
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    zero, one = torch.zeros((1, 8), device="cuda"), torch.ones((1, 8), device="cuda")
    da, dwg, dwu = moe.gmm_glu_bwd(one, zero, one, x, w, w, off, act=moe.ACT_RELU)
    assert not da.any() and not dwg.any() and not dwu.any()


def test_fused_halves_off_16_bytes_are_refused():
    """One (e,Hin,2N) tensor whose up half does not start on 16 bytes."""
    w = torch.zeros((1, 8, 2 * 260), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    with pytest.raises(moe.MoeError) as ei:
        moe.gmm_glu(x, w[:, :, :260], w[:, :, 260:], off)
    assert ei.value.status == moe.ERR_MISALIGNED


def test_no_rows():
    """A = 0: the forward pass does nothing, weight gradients are zeros."""
    w = torch.randn((3, 64, 32), device="cuda").to(torch.bfloat16)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert moe.gmm_glu(x, w, w, off).shape == (0, 32)
    e = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    dw = [torch.full((3, 64, 32), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    da, dwg, dwu = moe.gmm_glu_bwd(e, e, e, x, w, w, off, dw_gate=dw[0], dw_up=dw[1])
    assert da.shape == (0, 64) and not dwg.any() and not dwu.any()
    assert not moe.gmm_wgrad(x, e, off, out=dw[2]).any()
    assert moe.gmm_dgrad(e, w, off).shape == (0, 64)


@pytest.mark.parametrize("dt", list(DT))
def test_gather_entries_out_of_range_read_as_zero_rows(dt):
    c = Case([200, 70], 64, 64, dt, 3, gather=True)
    rows = c.rows.clone()
    bad = torch.tensor([0, 5, 199, 201, 269])
    rows[bad] = torch.tensor([-1, 2 ** 31 - 1, c.x.shape[0] * c.div, -2 ** 31, -7], dtype=torch.int32, device="cuda")
    c.rows = rows
    c.xr[bad] = 0.0
    check_glu(c, "silu")
    check_bwd(c, "silu")


def test_values_of_other_experts_do_not_leak():
    """NaN and infinity in one expert's rows and weights stay with it: the rows
    behind a partial tile belong to the next expert."""
    c = Case([70, 300, 5], 72, 40, "bf16", 11, gather=False)
    clean = moe.gmm_glu(c.x, c.wg, c.wu, c.offsets)
    args = [t.cuda() for t in (c.dout, c.gate, c.up)]
    grads = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets)
    x, wg, wu = c.x.clone(), c.wg.clone(), c.wu.clone()
    x[70:370] = float("nan")
    wg[1], wu[1] = float("inf"), float("nan")
    args2 = [t.clone() for t in args]
    for t in args2:
        t[70:370] = float("inf")
    out = moe.gmm_glu(x, wg, wu, c.offsets)
    bad = moe.gmm_glu_bwd(*args2, x, wg, wu, c.offsets)
    keep = torch.cat([torch.arange(0, 70), torch.arange(370, 375)]).cuda()
    assert torch.equal(out[keep], clean[keep]) and torch.equal(bad[0][keep], grads[0][keep])
    for i in (1, 2):
        for e in (0, 2):
            assert torch.equal(bad[i][e], grads[i][e])
    assert torch.isnan(out[70:370]).all()


@pytest.mark.parametrize("name", ["decode", "tiles_many", "odd_many", "long_dense", "f32_ragged", "f32_split",
                                  "f32_one_wide", "f32_odd_many", "five_by_seven", "long_odd", "long_odd_f32"])
def test_rows_outside_and_other_experts_change_nothing(name):
    """Experts that start behind the first rows; NaN and infinities in the rows that
    no expert covers and in one expert's own: every other expert's results keep
    their bits, and rows without an expert stay as they were."""
    counts, Hin, N, dt, _, fused, _ = GLU_CASES[name]
    front, tail = 3, 2
    counts = list(counts) if len(counts) > 1 else [counts[0] - 40, 40]
    c = Case([front, *counts], Hin, N, dt, 5, gather=False, fused=fused, tail=tail)
    e, off = len(counts), c.off[1:].copy()
    offsets = torch.from_numpy(off).cuda()
    wg, wu = (w[1:].clone(memory_format=torch.contiguous_format) for w in (c.wg, c.wu))
    bad = next(i for i in range(e - 1, -1, -1) if counts[i] > 0)
    own = [c.x, *(t.cuda() for t in (c.dout, c.gate, c.up))]

    def run(x, dout, gate, up):
        new = lambda n: torch.full((c.A, n), 7.0, dtype=c.dt, device="cuda")  # noqa: E731
        out, da, da1 = new(N), new(Hin), new(Hin)
        moe.gmm_glu(x, wg, wu, offsets, out=out)
        _, dwg, dwu = moe.gmm_glu_bwd(dout, gate, up, x, wg, wu, offsets, da=da)
        moe.gmm_dgrad(dout, wg, offsets, out=da1)
        return (out, da, da1), (dwg, dwu, moe.gmm_wgrad(x, dout, offsets))

    rows, weights = run(*own)
    for t in rows:
        assert bool((t[:front] == 7.0).all()) and bool((t[int(off[-1]):] == 7.0).all())
    for t in own:
        t[0], t[1, ::2], t[2], t[-1], t[-2, ::3] = float("nan"), float("inf"), -float("inf"), float("nan"), float("inf")
    again, weights2 = run(*own)
    for a, b in zip((*rows, *weights), (*again, *weights2)):
        assert torch.equal(a, b)
    for t in own:
        t[int(off[bad])] = float("nan")
        t[int(off[bad + 1]) - 1, ::2] = float("inf")
    again, weights2 = run(*own)
    keep = torch.ones(c.A, dtype=torch.bool, device="cuda")
    keep[int(off[bad]):int(off[bad + 1])] = False
    for a, b in zip(rows, again):
        assert torch.equal(a[keep], b[keep])
    others = [i for i in range(e) if i != bad]
    for a, b in zip(weights, weights2):
        assert torch.equal(a[others], b[others])


def test_gated_outputs_and_gradients_are_bitwise_stable():
    c = case_of("tiles_many")
    args = [t.cuda() for t in (c.dout, c.gate, c.up)]

    def once():
        return [moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)[:int(c.off[-1])],
                *moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)]

    a = once()
    for _ in range(3):
        b = once()
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
        assert torch.equal(a[1][:int(c.off[-1])], b[1][:int(c.off[-1])])


def test_gradient_parts_alone_equal_both():
    c = case_of("tiles_fold")
    args = [t.cuda() for t in (c.dout, c.gate, c.up)]
    n = int(c.off[-1])
    da, dwg, dwu = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)
    one = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div, need_dw=False)
    two = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div, need_da=False)
    assert one[1] is None and one[2] is None and two[0] is None
    assert torch.equal(one[0][:n], da[:n]) and torch.equal(two[1], dwg) and torch.equal(two[2], dwu)


def test_strided_gradients_leave_the_gap():
    """Weight gradients written as column ranges of a wider tensor."""
    c = case_of("tiles")
    args = [t.cuda() for t in (c.dout, c.gate, c.up)]
    _, dwg, dwu = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)
    wide = torch.full((c.e, c.Hin, 2 * c.N + 32), 7.0, dtype=c.dt, device="cuda")
    g, u = wide[:, :, 8:8 + c.N], wide[:, :, c.N + 16:2 * c.N + 16]
    moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div, dw_gate=g, dw_up=u)
    assert torch.equal(g, dwg) and torch.equal(u, dwu)
    for a, b in ((0, 8), (8 + c.N, c.N + 16), (2 * c.N + 16, 2 * c.N + 32)):
        assert bool((wide[:, :, a:b] == 7.0).all())


def test_gated_layer_forward_and_backward_through_the_router():
    """route -> permute -> gmm_glu (gathered) -> moe_gmm -> combine, and its
    gradients for tokens and expert weights, against fp64 on the GPU's own
    selection. Each bf16 intermediate is off by up to 2^-8 of its value, which
    the sums average: normwise 2e-2, the library's bf16 bar."""
    T, H, E, K, F = 300, 128, 8, 2, 192
    gen = torch.Generator().manual_seed(0)
    mk = lambda *s, f=1.0: (torch.randn(s, generator=gen) * f).to(torch.bfloat16)  # noqa: E731
    x, wr = mk(T, H), mk(H, E, f=H ** -0.5)
    wg, wu, wd = mk(E, H, F, f=H ** -0.5), mk(E, H, F, f=H ** -0.5), mk(E, F, H, f=F ** -0.5)
    dy = mk(T, H)
    X, WR, WG, WU, WD, DY = (t.cuda() for t in (x, wr, wg, wu, wd, dy))
    idx, gates = moe.route(X, WR, K)
    p = moe.permute(idx, E)
    hid, g, u = moe.gmm_glu(X, WG, WU, p["offsets"], rows=p["perm_src"], row_div=K, save=True)
    yp = moe.gmm(hid, WD, p["offsets"])
    y = moe.combine(yp, p["perm_dst"], gates, T, K)
    # backward: rows of the down projection's output gradient are gate * dy
    src = p["perm_src"].long()
    dyp = (gates.reshape(-1)[src, None] * DY[src // K].float()).to(torch.bfloat16)
    dhid = moe.gmm_dgrad(dyp, WD, p["offsets"])
    dwd = moe.gmm_wgrad(hid, dyp, p["offsets"])
    da, dwg, dwu = moe.gmm_glu_bwd(dhid, g, u, X, WG, WU, p["offsets"], rows=p["perm_src"], row_div=K)
    dx = moe.combine(da, p["perm_dst"], torch.ones((T, K), device="cuda"), T, K)
    torch.cuda.synchronize()

    lv = [t.double().requires_grad_() for t in (x, wg, wu, wd)]
    ids, gt = idx.cpu().long(), gates.cpu().double()
    ref = torch.zeros((T, H), dtype=torch.float64)
    for k in range(K):
        for e in range(E):
            t = torch.nonzero(ids[:, k] == e)[:, 0]
            h = lv[0][t] @ lv[1][e]
            h = h * torch.sigmoid(h) * (lv[0][t] @ lv[2][e])
            ref = ref.index_add(0, t, gt[t, k, None] * (h @ lv[3][e]))
    ref.backward(dy.double())
    for name, got, want in (("y", y, ref.detach()), ("dx", dx, lv[0].grad), ("dwg", dwg, lv[1].grad),
                            ("dwu", dwu, lv[2].grad), ("dwd", dwd, lv[3].grad)):
        err = (got.cpu().double() - want).abs().max() / want.abs().max()
        assert err <= 2e-2, f"{name}: {err:.3e}"


def test_graph_replays_match_eager():
    """Forward and backward captured in one graph, replayed on new inputs with
    eager work between the replays."""
    c = case_of("tiles_many")
    c2 = Case(c.counts, c.Hin, c.N, "bf16", 99, gather=True, tail=7, T=c.x.shape[0])
    args = [t.cuda() for t in (c.dout, c.gate, c.up)]
    n = int(c.off[-1])

    def step():
        out = moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)
        return [out, *moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x0 = c.x.clone()
    for k in range(4):
        c.x.copy_(x0 if k % 2 == 0 else c2.x)
        now = want if k % 2 == 0 else [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b, rows in zip(got, now, (n, n, None, None)):
            assert torch.equal(a[:rows], b[:rows])


@pytest.mark.parametrize("name", ["f32_ragged", "f32_split", "odd_many", "long_odd"])
def test_more_graph_replays_match_eager(name):
    c = case_of(name)
    args = [t.cuda() for t in (c.dout, c.gate, c.up)]
    n = int(c.off[-1])

    def step():
        out = moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)
        grads = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)
        return [out[:n], grads[0][:n], *grads[1:], moe.gmm_dgrad(args[0], c.wg, c.offsets)[:n],
                moe.gmm_wgrad(c.x, args[0], c.offsets, rows=c.rows, row_div=c.div)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(4):
        c.x.mul_(-0.5 if k % 2 else 1.0)
        now = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, now):
            assert torch.equal(a, b)


def test_call_on_another_stream():
    """stream=: the launch and the buffers the call allocates belong to it."""
    c = case_of("tiles")
    want = moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)
    args = [t.cuda() for t in (c.dout, c.gate, c.up)]
    wantb = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div, stream=s)
    gotb = moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    for a, b in zip(gotb, wantb):
        assert torch.equal(a, b)


@pytest.mark.parametrize("N", [2112, 2113])
def test_rows_beyond_32_bit_offsets(N):
    """More than 2^31 elements and 2^32 bytes in every row matrix: the last
    expert's rows against a call on those rows alone (the same sums)."""
    A, Hin, tail = 1 << 20, 64, 300
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((A, Hin), generator=gen, device="cuda").to(torch.bfloat16)
    wg, wu = ((torch.randn((3, Hin, N), generator=gen, device="cuda") / 8).to(torch.bfloat16) for _ in range(2))
    off = torch.tensor([0, 5, A - tail, A], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 0, 0, tail], dtype=torch.int32, device="cuda")
    last = slice(A - tail, A)
    out, gate, up = moe.gmm_glu(x, wg, wu, off, save=True)
    assert out.numel() > 2 ** 31
    ref = moe.gmm_glu(x[last].clone(), wg, wu, one, save=True)
    h = half_step(torch.bfloat16)
    for a, b in zip((out, gate, up), ref):
        a, b = a[last].double(), b.double()
        # the two calls may take other tiles: binary32 sums of 64 terms in another order
        assert bool(((a - b).abs() <= 2 * h * b.abs() + 2.0 ** -12).all())
    dout = torch.randn((A, N), generator=gen, device="cuda", dtype=torch.bfloat16)
    da, dwg, dwu = moe.gmm_glu_bwd(dout, gate, up, x, wg, wu, off)
    rda, rdg, rdu = moe.gmm_glu_bwd(dout[last].clone(), gate[last].clone(), up[last].clone(), x[last].clone(), wg, wu, one)
    for a, b in ((da[last], rda), (dwg[2], rdg[2]), (dwu[2], rdu[2])):
        err = (a.double() - b.double()).abs().max() / b.double().abs().max()
        assert err <= 2 * h
    del out, gate, up, da
    # a gradient for rows of N columns, and one over 2^20 rows of it
    w = wg.transpose(1, 2).contiguous()  # (3, N, Hin)
    dl = torch.randn((A, Hin), generator=gen, device="cuda", dtype=torch.bfloat16)
    got = moe.gmm_dgrad(dl, w, off)[last]
    assert bool((got.double() - moe.gmm_dgrad(dl[last].clone(), w, one).double()).abs().max() <= 2 * h * got.double().abs().max())
    dw = moe.gmm_wgrad(dout, dl, off)
    want = moe.gmm_wgrad(dout[last].clone(), dl[last].clone(), one)
    assert bool((dw[2].double() - want[2].double()).abs().max() <= 2 * h * want[2].double().abs().max())


def test_two_streams_at_once():
    """Calls on two streams share nothing: each result equals its own."""
    a, b = case_of("tiles_many"), case_of("long_gathered")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def go(c, s):
        args = [t.cuda() for t in (c.dout, c.gate, c.up)]
        torch.cuda.synchronize()
        return lambda: [moe.gmm_glu(c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div, stream=s),
                        *moe.gmm_glu_bwd(*args, c.x, c.wg, c.wu, c.offsets, rows=c.rows, row_div=c.div, stream=s)]

    calls = [go(a, streams[0]), go(b, streams[1])]
    want = []
    for f in calls:
        want.append([t.clone() for t in f()])
        torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, f in enumerate(calls):
            got[i].append(f())
    torch.cuda.synchronize()
    for i, c in enumerate((a, b)):
        n = int(c.off[-1])
        for r in got[i]:
            for x, y, rows in zip(r, want[i], (n, n, None, None)):
                assert torch.equal(x[:rows], y[:rows])
