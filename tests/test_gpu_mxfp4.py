"""MXFP4 quantisers (bit-exact against the recipe in fp64) and the grouped product
that quantises its rows (against fp64 sums of the same codes)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_06_amd as moe
import synth
from tests.helpers import to_dev

pytestmark = pytest.mark.gpu

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def as_dt(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16 if dt == "bf16" else torch.float32)


def recipe(x64, axis):
    """(packed codes, scale bytes, values) of finite fp64 x by brute force: the
    nearest grid value among all, ties to the even code."""
    b = np.moveaxis(x64, axis, -1)
    b = b.reshape(b.shape[:-1] + (-1, 32))
    top = np.abs(b).max(-1)
    ex = np.frexp(top)[1] - 1 - 2  # frexp: top = m 2^e, m in [1/2, 1)
    ex = np.where(top > 0, np.clip(ex, -127, 127), 0)
    v = np.abs(b) / np.ldexp(1.0, ex)[..., None]
    dist = np.abs(v[..., None] - GRID)
    best = dist.min(-1, keepdims=True)
    # of the nearest (one or two codes) the even one
    cand = dist == best
    order = np.where(cand, np.where(np.arange(8) % 2 == 0, 0, 1), 9)
    code = order.argmin(-1)
    vals = np.copysign(GRID[code], b) * np.ldexp(1.0, ex)[..., None]
    full = (code | (np.signbit(b) << 3)).astype(np.uint8).reshape(b.shape[:-2] + (-1,))
    packed = full[..., 0::2] | (full[..., 1::2] << 4)
    back = lambda a: np.ascontiguousarray(np.moveaxis(a, -1, axis))  # noqa: E731
    return back(packed), back((ex + 127).astype(np.uint8)), back(vals.reshape(full.shape))


def hard_rows(R, H, dt, seed):
    """Rows with blocks of very unequal magnitude, zeros, ties, grid points,
    saturating values and subnormals."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, H)) * np.exp2(rng.integers(-20, 20, (R, H // 32))).repeat(32, 1)
    b = x.reshape(R, H // 32, 32)
    kinds = [lambda n: np.zeros(n), lambda n: rng.choice(np.concatenate([GRID, -GRID]), n),
             lambda n: rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.9, 7.9], n) * rng.choice([-1, 1], n),
             lambda n: rng.standard_normal(n) * 2.0 ** -126, lambda n: rng.standard_normal(n) * 2.0 ** -131,
             lambda n: rng.standard_normal(n) * 2.0 ** 125, lambda n: np.where(np.arange(n) == 5, -2.0 ** 127 * 1.9, 1.0),
             lambda n: np.where(np.arange(n) == 31, 1.0, -1e-30)]
    for i in range(R * (H // 32)):
        if i % 3 == 0:
            b[i // (H // 32), i % (H // 32)] = kinds[(i // 3) % len(kinds)](32)
    return as_dt(b.reshape(R, H), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,H", [(1, 256), (15, 512), (16, 256), (17, 1280), (100, 768), (3, 7168)])
def test_rows_bit_exact(dt, R, H):
    x = hard_rows(R, H, dt, R * H)
    q, sc, vals = moe.quant_mxfp4_rows(x.cuda(), values=True)
    q0, sc0 = moe.quant_mxfp4_rows(x.cuda())
    none = moe.quant_mxfp4_rows(x.cuda(), codes=False, values=True)
    torch.cuda.synchronize()
    wq, ws, wv = recipe(x.double().numpy(), 1)
    assert np.array_equal(sc.cpu().numpy(), synth.mx_scales_slice_major(ws, 8))
    assert np.array_equal(q.cpu().numpy(), wq)
    assert np.array_equal(vals.double().cpu().numpy(), wv)
    assert torch.equal(q0, q) and torch.equal(sc0, sc)
    assert none[0] is None and none[1] is None and torch.equal(none[2].view(torch.int16), vals.view(torch.int16))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("e,Hin,N", [(1, 256, 16), (2, 512, 80), (3, 256, 64), (1, 768, 1040)])
def test_weights_bit_exact(dt, e, Hin, N):
    w = hard_rows(e * N, Hin, dt, N).reshape(e, N, Hin).transpose(1, 2).contiguous()
    q, sc, vals = moe.quant_mxfp4_weights(w.cuda(), values=True)
    q0, sc0 = moe.quant_mxfp4_weights(w.cuda())
    none = moe.quant_mxfp4_weights(w.cuda(), codes=False, values=True)
    torch.cuda.synchronize()
    wq, ws, wv = recipe(w.double().numpy(), 1)
    assert np.array_equal(sc.cpu().numpy(), synth.mx_weight_scales_interleaved(ws))
    assert np.array_equal(q.cpu().numpy(), wq)
    assert np.array_equal(vals.double().cpu().numpy(), wv)
    assert torch.equal(q0, q) and torch.equal(sc0, sc)
    assert torch.equal(none[2].view(torch.int16), vals.view(torch.int16))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_non_finite_blocks_are_nan(dt):
    x = as_dt(np.random.default_rng(0).standard_normal((4, 512)), dt)
    clean = moe.quant_mxfp4_rows(x.cuda(), values=True)
    for r, h, v in ((0, 5, float("nan")), (1, 64, float("inf")), (2, 511, -float("inf")), (2, 100, float("nan"))):
        x[r, h] = v
    q, sc, vals = (t.cpu() for t in moe.quant_mxfp4_rows(x.cuda(), values=True))
    byte = sc.permute(1, 0, 2).reshape(4, 16)
    hit = torch.zeros((4, 16), dtype=torch.bool)
    for r, h in ((0, 5), (1, 64), (2, 511), (2, 100)):
        hit[r, h // 32] = True
    wide = hit.repeat_interleave(32, 1)
    assert bool((byte[hit] == 255).all()) and bool(torch.isnan(vals[wide]).all())
    assert bool((q[hit.repeat_interleave(16, 1)] == 0).all())
    for got, want in ((vals[~wide], clean[2].cpu()[~wide]), (q[~hit.repeat_interleave(16, 1)], clean[0].cpu()[~hit.repeat_interleave(16, 1)]),
                      (byte[~hit], clean[1].cpu().permute(1, 0, 2).reshape(4, 16)[~hit])):
        assert torch.equal(got, want)
    w = x.t().contiguous()[None].repeat(1, 1, 4)  # (1, 512, 16)
    wq, wsc, wv = (t.cpu() for t in moe.quant_mxfp4_weights(w.cuda(), values=True))
    assert torch.equal(torch.isnan(wv[0, :, :4]), wide.t())


def test_rows_gather():
    x = hard_rows(9, 512, "bf16", 1).cuda()
    src = torch.tensor([0, 26, 5, 27, -1, 2 ** 31 - 1, 3, 3, 13] * 5, dtype=torch.int32, device="cuda")
    q, sc, v = moe.quant_mxfp4_rows(x, rows=src, row_div=3, values=True)
    t = torch.div(src, 3, rounding_mode="floor")
    ok = (src >= 0) & (t < 9)
    xr = torch.where(ok[:, None], x[t.clamp(0, 8).long()], torch.zeros((), dtype=x.dtype, device="cuda"))
    q1, sc1, v1 = moe.quant_mxfp4_rows(xr, values=True)
    assert torch.equal(q, q1) and torch.equal(sc, sc1) and torch.equal(v.view(torch.int16), v1.view(torch.int16))
    assert bool((sc.permute(1, 0, 2)[~ok] == 127).all())


def _values_of(codes, axis):
    c = np.moveaxis(codes, axis, -1)
    full = np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (-1,))
    v = GRID[full & 7] * np.where(full & 8, -1.0, 1.0)
    return np.moveaxis(v, -1, axis)


# counts, Hin, N, type of x, gather, rows behind the last expert
DYN = {
    "one_row": ([1], 256, 16, "bf16", False, 0),
    "one_row_gather_f32": ([1], 512, 32, "f32", True, 0),
    "decode": ([0, 1, 3, 0, 2, 16, 1], 4096, 96, "bf16", True, 0),
    "decode_f32": ([2, 0, 5], 768, 208, "f32", True, 1),
    "decode_17": ([17, 0, 33], 1024, 272, "bf16", True, 2),
    "decode_48": ([48, 49, 1], 512, 144, "bf16", False, 0),
    "decode_k_odd": ([4, 3], 1280, 128, "bf16", True, 0),
    "skewed": ([1, 0, 200, 2, 0, 1, 1, 1, 1, 1], 256, 80, "bf16", True, 3),
    "decode_16_one": ([16], 512, 272, "bf16", False, 0),
    "decode_16_spread": ([3, 13], 512, 48, "f32", True, 0),
    "tiles": ([256, 0, 300, 129], 512, 272, "bf16", True, 5),
    "tiles_f32": ([500], 256, 64, "f32", False, 0),
}


@pytest.mark.parametrize("act", [moe.ACT_NONE, moe.ACT_RELU], ids=["none", "relu"])
@pytest.mark.parametrize("name", list(DYN))
def test_dyn_product(name, act):
    """Products of two E2M1 values and powers of two are exact; a binary32 sum of
    Hin of them is off by at most Hin * 2^-23 * sum|products|, and the bf16 result
    by half a step, 2^-8."""
    counts, Hin, N, dt, gather, tail = DYN[name]
    rng = np.random.default_rng(sum(map(ord, name)))
    e, A = len(counts), sum(counts) + tail
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = max(1, A // 2) if gather else A
    x = hard_rows(T, Hin, "bf16", A)
    x = torch.where(x.float().abs() > 2.0 ** 40, torch.ones((), dtype=x.dtype), x)  # finite sums
    x = x.to(torch.bfloat16 if dt == "bf16" else torch.float32)
    rows = rng.integers(0, T * 3, A).astype(np.int32) if gather else None
    w = as_dt(rng.standard_normal((e, Hin, N)) * Hin ** -0.5, "f32").cuda()
    q, sw, wv = moe.quant_mxfp4_weights(w, values=True)
    out = torch.full((A, N), 7.0, dtype=torch.bfloat16, device="cuda")
    offs = to_dev(off)
    xd, rd = x.cuda(), None if rows is None else to_dev(rows)
    moe.gmm_mxfp4_dyn(xd, q, sw, offs, act=act, rows=rd, row_div=3, out=out)
    again = moe.gmm_mxfp4_dyn(xd, q, sw, offs, act=act, rows=rd, row_div=3)
    aq, asc = moe.quant_mxfp4_rows(xd, rows=rd, row_div=3)
    two = moe.gmm_mxfp4(aq, asc, q, sw, offs, act=act)
    torch.cuda.synchronize()
    n = int(off[-1])
    assert torch.equal(again[:n], out[:n])
    assert bool((out[n:] == 7.0).all())
    xv = recipe(x.double().numpy(), 1)[2]
    xv = xv if rows is None else xv[rows // 3]
    wv = wv.double().cpu().numpy()
    for i in range(e):
        s = slice(off[i], off[i + 1])
        want, mag = xv[s] @ wv[i], np.abs(xv[s]) @ np.abs(wv[i])
        b = Hin * 2.0 ** -23 * mag
        if act == moe.ACT_RELU:
            want = np.maximum(want, 0)
        for got in (out, two):
            err = np.abs(got[s].double().cpu().numpy() - want)
            lim = b + 2.0 ** -8 * (np.abs(want) + b)
            assert (err <= lim).all(), f"expert {i}: off by up to {(err - lim).max():.3e} beyond the bound"


@pytest.mark.parametrize("Hin,gather", [(256, True), (768, False), (1280, True)])
def test_product_on_large_tiles(Hin, gather):
    """Many rows and columns, so that 256-row tiles are taken: whole ones, ones
    with up to 32 rows riding along, short ones; the last columns part of a tile.
    Bounds as above; an expert by itself, on 128-row tiles, gives the same bits
    (the same products in the same order of additions)."""
    counts = [256, 257, 0, 288, 289, 512, 544, 545, 1, 30, 700, 255, 800]
    N, e, A = 2064, len(counts), sum(counts) + 4
    rng = np.random.default_rng(Hin)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = 900 if gather else A
    x = as_dt(rng.standard_normal((T, Hin)), "bf16")
    rows = rng.integers(0, 2 * T, A).astype(np.int32) if gather else None
    q, sw, wv = moe.quant_mxfp4_weights(as_dt(rng.standard_normal((e, Hin, N)), "bf16").cuda(), values=True)
    out = torch.full((A, N), 7.0, dtype=torch.bfloat16, device="cuda")
    rd = None if rows is None else to_dev(rows)
    moe.gmm_mxfp4_dyn(x.cuda(), q, sw, to_dev(off), rows=rd, row_div=2, out=out)
    aq, asc = moe.quant_mxfp4_rows(x.cuda(), rows=rd, row_div=2)
    two = moe.gmm_mxfp4(aq, asc, q, sw, to_dev(off))
    n = int(off[-1])
    assert torch.equal(two[:n], out[:n])
    assert bool((out[n:] == 7.0).all())
    xv = recipe(x.double().numpy(), 1)[2]
    xv = torch.from_numpy(xv if rows is None else xv[rows // 2]).cuda()
    for i in range(e):
        s = slice(int(off[i]), int(off[i + 1]))
        w = wv[i].double()
        want, mag = xv[s] @ w, xv[s].abs() @ w.abs()
        b = Hin * 2.0 ** -23 * mag
        assert bool(((out[s].double() - want).abs() <= b + 2.0 ** -8 * (want.abs() + b)).all()), f"expert {i}"
        if counts[i] > 0:
            one = torch.tensor([0, counts[i]], dtype=torch.int32, device="cuda")
            alone = moe.gmm_mxfp4(aq[s].clone(), asc[:, s].clone(memory_format=torch.contiguous_format), q[i:i + 1], sw[i:i + 1], one)
            assert torch.equal(alone, out[s]), f"expert {i} alone"


@pytest.mark.parametrize("A", [3, 40, 300])
def test_dyn_non_finite_rows_stay_alone(A):
    x = hard_rows(A, 512, "bf16", 2).float().clamp(-1e6, 1e6).to(torch.bfloat16)
    w = torch.randn((1, 512, 64), generator=torch.Generator().manual_seed(0)).cuda()
    q, sw = moe.quant_mxfp4_weights(w)
    off = torch.tensor([0, A], dtype=torch.int32, device="cuda")
    clean = moe.gmm_mxfp4_dyn(x.cuda(), q, sw, off)
    x[1, 77] = float("nan")
    x[2, 300] = float("inf")
    out = moe.gmm_mxfp4_dyn(x.cuda(), q, sw, off)
    keep = torch.tensor([r for r in range(A) if r not in (1, 2)], device="cuda")
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[1:3]).all())


@pytest.mark.parametrize("counts,Hin,N", [([1, 3, 2], 512, 96), ([40, 70, 30], 768, 272),
                                          ([300, 1, 290, 2000, 800, 700], 512, 2064)],
                         ids=["streamed", "small_tiles", "large_tiles"])
def test_rows_outside_and_other_experts_change_nothing(counts, Hin, N):
    """Experts that start behind the first rows; NaN in rows that no expert covers
    and in the last expert's: the others keep their bits."""
    front, tail, e = 2, 3, len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + front
    A = int(off[-1]) + tail
    gen = torch.Generator().manual_seed(A)
    x = torch.randn((A, Hin), generator=gen).to(torch.bfloat16).cuda()
    q, sw = moe.quant_mxfp4_weights(torch.randn((e, Hin, N), generator=gen).cuda())

    def run():
        out, two = (torch.full((A, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        moe.gmm_mxfp4_dyn(x, q, sw, to_dev(off), out=out)
        moe.gmm_mxfp4(*moe.quant_mxfp4_rows(x), q, sw, to_dev(off), out=two)
        return out, two

    clean = run()
    for t in clean:
        assert bool((t[:front] == 7.0).all()) and bool((t[A - tail:] == 7.0).all())
    assert torch.equal(*clean)
    x[:front], x[A - tail:] = float("nan"), float("inf")
    for a, b in zip(clean, run()):
        assert torch.equal(a, b)
    x[int(off[-2]):int(off[-1])] = float("nan")
    for a, b in zip(clean, run()):
        assert torch.equal(a[:int(off[-2])], b[:int(off[-2])])
        assert bool(torch.isnan(b[int(off[-2]):int(off[-1])]).all())


def test_mxfp4_expert_ffn_end_to_end():
    """Weights and rows quantised on the device, two products, combine: against
    fp64 sums over codes of the recipe in fp64, the hidden rows
    those the device produced. Normwise 2e-2, the library's bf16 bar."""
    T, H, E, K, F = 40, 512, 8, 2, 256
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    wr = (torch.randn((H, E), generator=gen) * H ** -0.5).to(torch.bfloat16).cuda()
    w1, w2 = (torch.randn((E, a, b), generator=gen) * a ** -0.5 for a, b in ((H, F), (F, H)))
    q1, s1 = moe.quant_mxfp4_weights(w1.cuda())
    q2, s2 = moe.quant_mxfp4_weights(w2.to(torch.bfloat16).cuda())
    idx, gate = moe.route(x, wr, K)
    p = moe.permute(idx, E)
    h = moe.gmm_mxfp4_dyn(x, q1, s1, p["offsets"], act=moe.ACT_RELU, rows=p["perm_src"], row_div=K)
    yp = moe.gmm_mxfp4_dyn(h, q2, s2, p["offsets"])
    y = moe.combine(yp, p["perm_dst"], gate, T, K)
    torch.cuda.synchronize()
    src = p["perm_src"].cpu().numpy()
    off = p["offsets"].cpu().numpy()
    a1, b1, _ = recipe(x.double().cpu().numpy()[src // K], 1)
    a2, b2, _ = recipe(h.double().cpu().numpy(), 1)
    k1, c1, _ = recipe(w1.double().numpy(), 1)
    k2, c2, _ = recipe(w2.to(torch.bfloat16).double().numpy(), 1)
    h0 = np.maximum(_grouped(a1, b1, k1, c1, off), 0)
    y0 = _grouped(a2, b2, k2, c2, off)
    assert np.abs(h.double().cpu().numpy() - h0).max() <= 2e-2 * np.abs(h0).max()
    assert np.abs(yp.double().cpu().numpy() - y0).max() <= 2e-2 * np.abs(y0).max()
    dst, g = p["perm_dst"].cpu().numpy().reshape(T, K), gate.double().cpu().numpy()
    want = (g[:, :, None] * y0[dst]).sum(1)
    assert np.abs(y.double().cpu().numpy() - want).max() <= 2e-2 * np.abs(want).max()


def _grouped(a, sa, w, sw, off):
    A = _values_of(a, 1) * np.exp2(sa.astype(np.float64) - 127).repeat(32, 1)
    W = _values_of(w, 1) * np.exp2(sw.astype(np.float64) - 127).repeat(32, 1)
    return np.concatenate([A[off[i]:off[i + 1]] @ W[i] for i in range(len(off) - 1)])


def test_graph_replays_match_eager():
    x = hard_rows(50, 512, "bf16", 4).float().clamp(-1e6, 1e6).to(torch.bfloat16).cuda()
    w = torch.randn((4, 512, 96), device="cuda")
    off = torch.tensor([0, 7, 7, 31, 50], dtype=torch.int32, device="cuda")

    def step():
        q, sw, v = moe.quant_mxfp4_weights(w, values=True)
        return [q, sw, v, moe.gmm_mxfp4_dyn(x, q, sw, off)]

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(4):
        x.copy_(x.flip(0))
        w.mul_(-1.5)
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_on_another_stream():
    x = hard_rows(50, 512, "bf16", 4).float().clamp(-1e6, 1e6).to(torch.bfloat16).cuda()
    w = torch.randn((1, 512, 96), device="cuda")
    off = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    q, sw = moe.quant_mxfp4_weights(w)
    want = moe.gmm_mxfp4_dyn(x, q, sw, off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q2, sw2 = moe.quant_mxfp4_weights(w, stream=s)
    got = moe.gmm_mxfp4_dyn(x, q2, sw2, off, stream=s)
    s.synchronize()
    assert torch.equal(q, q2) and torch.equal(sw, sw2) and torch.equal(got, want)


def test_rows_and_weights_beyond_32_bit_offsets():
    """More than 2^31 values (2^32 bytes): the last rows and the last expert
    against calls on those alone, bit for bit."""
    R, H = 300_001, 7168
    x = torch.randn((R, H), device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 2 ** 31
    q, sc, v = moe.quant_mxfp4_rows(x, values=True)
    q1, sc1, v1 = moe.quant_mxfp4_rows(x[-33:].clone(), values=True)
    assert torch.equal(q[-33:], q1) and torch.equal(sc[:, -33:], sc1) and torch.equal(v[-33:], v1)
    # a product gathering rows from both ends of x
    w, sw = moe.quant_mxfp4_weights(torch.randn((2, H, 32), device="cuda"))
    off = torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda")
    rows = torch.tensor([R - 1, 0, R - 2, 5, R - 1, 1, R - 33], dtype=torch.int32, device="cuda")
    got = moe.gmm_mxfp4_dyn(x, w, sw, off, rows=rows)
    assert torch.equal(got, moe.gmm_mxfp4_dyn(x[rows.long()], w, sw, off))
    del x, q, v
    w = torch.randn((160, 7168, 2048), device="cuda", dtype=torch.bfloat16)
    q, sc, v = moe.quant_mxfp4_weights(w, values=True)
    q1, sc1, v1 = moe.quant_mxfp4_weights(w[-1:].clone(), values=True)
    assert torch.equal(q[-1:], q1) and torch.equal(sc[-1:], sc1) and torch.equal(v[-1:], v1)
