"""Low-rank adapters and their gradients against plain fp64 computations (CPU, torch
double).

Tolerances, element by element, with S = 2^-23. A binary32 sum of n products is off by
n S of their magnitudes (one rounding of at most one step per addition; the products of
bf16 values are exact, fp32 ones round by half a step, counted in the same n). u and du
enter bf16 products as two bf16 terms, which leaves 2^-16 of each value out (fp32:
nothing). Bounds are sent through the second product with every value absolute; the
result's own rounding is half a step of its type (bf16 2^-8, fp32 2^-24)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_06_amd as moe
from test_gpu_ffn import DT, STEP, check, half_step

pytestmark = pytest.mark.gpu


class Case:
    """counts rows per adapter, `idle` listed rows behind them, T rows in all (those not
    listed at random places)."""

    def __init__(self, counts, H, N, R, dt, seed, idle=0, extra=0, scale=True, ordered=False):
        if ordered:  # without rows every row of the tensors is listed
            idle, extra = idle + extra, 0
        gen = torch.Generator().manual_seed(seed)
        self.counts, self.H, self.N, self.R, self.dt = list(counts), H, N, R, DT[dt]
        self.e, self.M = len(counts), sum(counts) + idle
        self.T = self.M + extra
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.offsets = torch.from_numpy(self.off).cuda()
        rows = torch.arange(self.M) if ordered else torch.randperm(self.T, generator=gen)[:self.M]
        self.rows = rows.long()
        self.rows_d = None if ordered else rows.to(torch.int32).cuda()
        mk = lambda *s, sc=1.0: (torch.randn(s, generator=gen) * sc).to(self.dt)  # noqa: E731
        self.x, self.base, self.dout, self.dx = mk(self.T, H), mk(self.T, N), mk(self.T, N), mk(self.T, H)
        self.a, self.b = mk(self.e, H, R, sc=H ** -0.5), mk(self.e, R, N, sc=0.3)
        self.scale = torch.rand((self.e,), generator=gen) * 2 - 0.5 if scale else None
        self.u = torch.randn((self.M, R), generator=gen)

    def dev(self, *names):
        return [getattr(self, n).cuda() if getattr(self, n) is not None else None for n in names]

    def segs(self):
        for e, (lo, hi) in enumerate(zip(self.off, self.off[1:])):
            s = float(self.scale[e].double()) if self.scale is not None else 1.0
            yield e, slice(int(lo), int(hi)), self.rows[int(lo):int(hi)], s

    @property
    def left_out(self):
        return 2.0 ** -16 if self.dt == torch.bfloat16 else 0.0

    def forward(self, **kw):
        x, a, b, scale = self.dev("x", "a", "b", "scale")
        return moe.lora(x, a, b, self.offsets, rows=self.rows_d, scale=scale, **kw)

    def check_forward(self, base=True):
        kept = torch.full((self.M, self.R), 7.0, device="cuda")
        given = self.base.cuda() if base else None
        out, u = self.forward(base=given, u=kept)
        assert u is kept
        start = self.base if base else torch.zeros_like(self.base)
        if base:
            assert torch.equal(given.cpu(), self.base)
        bare = self.forward(base=given)
        own = start.cuda().clone()
        self.forward(base=own, out=own)
        if not base:
            own_none = torch.full_like(own, 3.0)
            self.forward(out=own_none)
            assert (own_none.cpu()[self._others()] == 3).all()
            assert torch.equal(own_none.cpu()[self.rows], out.cpu()[self.rows])
        got = out.cpu()
        assert torch.equal(bare, out) and torch.equal(own, out)
        covered = int(self.off[-1])
        assert (u.cpu()[covered:] == 7).all()
        idle = torch.cat([self.rows[covered:], self._others()])
        assert torch.equal(got[idle], start[idle])
        h = half_step(self.dt)
        for e, s, t, f in self.segs():
            x, a, b = self.x[t].double(), self.a[e].double(), self.b[e].double()
            v, ev = x @ a, (self.H + 2) * STEP * (x.abs() @ a.abs())
            check(u[s], v, ev + 2.0 ** -24 * v.abs(), f"u of adapter {e}")
            ev = ev + (self.left_out + STEP) * v.abs()
            d, w = f * (v @ b), abs(f) * (v.abs() @ b.abs())
            bound = abs(f) * (ev @ b.abs()) + (2 * self.R + 4) * STEP * w
            want = start[t].double() + d
            bound = bound + STEP * want.abs()
            check(out[t], want, bound + h * (want.abs() + bound), f"out of adapter {e}")

    def _others(self):
        on = torch.zeros(self.T, dtype=torch.bool)
        on[self.rows] = True
        return (~on).nonzero()[:, 0]

    def check_backward(self, dw=None, base=True):
        dout, x, u, a, b, scale = self.dev("dout", "x", "u", "a", "b", "scale")
        given = self.dx.cuda() if base else None
        dwt = DT[dw] if dw else self.dt
        args = (dout, x, u, a, b, self.offsets)
        kw = dict(rows=self.rows_d, scale=scale, dw_dtype=dwt)
        dx, da, db = moe.lora_bwd(*args, base=given, **kw)
        start = self.dx if base else torch.zeros_like(self.dx)
        own = start.cuda().clone()
        parts = (moe.lora_bwd(*args, base=own, dx=own, need_da=False, need_db=False, **kw)[0],
                 moe.lora_bwd(*args, need_dx=False, need_db=False, **kw)[1],
                 moe.lora_bwd(*args, need_dx=False, need_da=False, **kw)[2])
        for one, whole in zip(parts, (dx, da, db)):
            assert torch.equal(one, whole)
        idle = torch.cat([self.rows[int(self.off[-1]):], self._others()])
        assert torch.equal(dx.cpu()[idle], start[idle])
        h, hw = half_step(self.dt), half_step(dwt)
        for e, s, t, f in self.segs():
            if not len(t):
                assert not da[e].any() and not db[e].any()
                continue
            d, xr, a64, b64 = self.dout[t].double(), self.x[t].double(), self.a[e].double(), self.b[e].double()
            du, w = f * (d @ b64.T), abs(f) * (d.abs() @ b64.abs().T)
            edu = (self.N + 4) * STEP * w + (self.left_out + STEP) * du.abs()
            g = du @ a64.T
            eg = edu @ a64.abs().T + (2 * self.R + 4) * STEP * (du.abs() @ a64.abs().T)
            want = start[t].double() + g
            eg = eg + STEP * want.abs()
            check(dx[t], want, eg + h * (want.abs() + eg), f"dx of adapter {e}")
            n = 2 * len(t) + 40  # rows, two terms each, and the joining of waves and parts
            g = xr.T @ du
            eg = xr.abs().T @ edu + n * STEP * (xr.abs().T @ du.abs())
            check(da[e], g, eg + hw * (g.abs() + eg), f"da of adapter {e}")
            v = self.u[s].double()
            g = f * (v.T @ d)
            eg = abs(f) * (n * STEP + self.left_out) * (v.abs().T @ d.abs())
            check(db[e], g, eg + hw * (g.abs() + eg), f"db of adapter {e}")


CASES = [
    # rows per adapter, H, N, R, type, more
    ([1], 16, 16, 1, "f32", {}), ([1], 4096, 4096, 16, "bf16", {}), ([3, 0, 1], 130, 70, 5, "bf16", dict(idle=2, extra=3)),
    ([2, 1, 0, 4], 64, 200, 8, "f32", dict(idle=1)), ([20, 0, 45], 256, 512, 16, "bf16", dict(idle=9, extra=5)),
    ([33, 17, 70], 1001, 501, 13, "bf16", dict(idle=3)), ([33, 17, 70], 1001, 501, 13, "f32", dict(extra=4)),
    ([300, 1, 140], 512, 768, 32, "bf16", dict(idle=70)), ([260, 129], 264, 520, 64, "bf16", dict(scale=False)),
    ([130, 300], 300, 300, 64, "f32", dict(idle=70)), ([200], 640, 384, 128, "bf16", {}), ([129], 200, 264, 100, "f32", {}),
    ([40, 30], 257, 259, 127, "bf16", dict(idle=1)), ([700, 400], 1024, 256, 16, "bf16", dict(ordered=True, extra=6)),
    ([500, 20, 0, 9, 700], 448, 320, 24, "f32", dict(ordered=True, idle=5)), ([1] * 70, 96, 1000, 33, "bf16", {}),
    ([5, 9, 3] * 40, 128, 64, 4, "f32", dict(idle=2)), ([0, 0], 64, 64, 8, "bf16", dict(idle=5)),
    ([1500], 4100, 72, 16, "bf16", {}), ([2100, 70], 40, 4097, 48, "bf16", dict(idle=1)), ([64], 8192, 40, 128, "f32", {}),
]


@pytest.mark.parametrize("counts,H,N,R,dt,more", CASES)
def test_forward(counts, H, N, R, dt, more):
    Case(counts, H, N, R, dt, H + N, **more).check_forward()


@pytest.mark.parametrize("counts,H,N,R,dt,more", CASES)
def test_backward(counts, H, N, R, dt, more):
    Case(counts, H, N, R, dt, H + N + 1, **more).check_backward()


MANY = [
    # tiles of 128 rows forwards, partial sums added first ([1700, ...]), tiles of 128 rows
    # backwards (over 2048 of them), rows in stretches ([2600, ...])
    ([600], 640, 384, 128, "bf16", {}), ([300, 1, 330], 512, 768, 32, "bf16", dict(idle=70)),
    ([530, 129], 264, 520, 64, "bf16", dict(scale=False)), ([330, 300], 300, 300, 64, "f32", dict(idle=70)),
    ([640], 200, 264, 100, "f32", {}), ([440, 130], 257, 259, 127, "bf16", dict(idle=1)),
    ([33, 517, 170], 1001, 501, 13, "bf16", dict(idle=3)), ([33, 517, 170], 1001, 501, 13, "f32", dict(extra=4)),
    ([1700, 1900], 4096, 264, 128, "bf16", dict(idle=2)), ([1700, 2000], 4100, 72, 128, "f32", {}),
    ([600, 77], 64, 4104, 48, "bf16", dict(idle=1)), ([700], 72, 4101, 20, "f32", {}),
    ([1200], 40, 5000, 128, "bf16", {}), ([513], 16, 4100, 8, "f32", {}),
    ([2100, 9, 0, 300], 136, 328, 64, "bf16", dict(idle=3)), ([1000, 1300], 72, 1037, 127, "bf16", {}),
    ([700, 1500], 264, 96, 20, "f32", dict(idle=70)), ([2600, 0, 500, 1], 520, 1032, 4, "bf16", dict(extra=3)),
    ([2600, 40], 257, 401, 3, "f32", {}),
]


@pytest.mark.parametrize("counts,H,N,R,dt,more", MANY)
def test_many_rows(counts, H, N, R, dt, more):
    Case(counts, H, N, R, dt, H + N + 2, **more).check_forward()
    Case(counts, H, N, R, dt, H + N + 3, **more).check_backward()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_without_a_shared_projection(dt):
    c = Case([70, 5], 136, 264, 16, dt, 1, idle=4, extra=3)
    c.check_forward(base=False)
    c.check_backward(dw="f32", base=False)


def test_long_sums_in_parts():
    """Rows and widths that split: 9000 rows of one adapter, 16000 wide."""
    Case([9000, 30], 128, 256, 8, "bf16", 2).check_backward(dw="f32")
    Case([40], 16000, 64, 8, "bf16", 3).check_forward()


def test_grouping_of_the_dispatch():
    """The grouping that moe_permute makes of each token's adapter, with E for none."""
    T, e = 500, 6
    gen = torch.Generator().manual_seed(4)
    adapter = torch.randint(0, e + 1, (T, 1), generator=gen, dtype=torch.int32)
    p = moe.permute(adapter.cuda(), e + 1)
    c = Case(torch.bincount(adapter[:, 0].long(), minlength=e + 1)[:e].tolist(), 192, 320, 16, "bf16", 5,
             idle=int((adapter == e).sum()))
    off = p["offsets"][:e + 1]
    rows = p["perm_src"]
    assert torch.equal(off.cpu(), c.offsets.cpu())
    c.rows, c.rows_d, c.offsets = rows.cpu().long(), rows, off
    c.check_forward()
    c.check_backward()


def test_rows_out_of_range():
    """Entries outside the tensors are passed over: nothing of them is read or written,
    and they add nothing to the adapters' gradients."""
    c = Case([40, 30], 96, 128, 8, "f32", 6, extra=2)
    gone = [3, 17, 45, 60]
    rows = c.rows.clone()
    rows[gone] = torch.tensor([-1, c.T, 2 ** 31 - 1, -2 ** 31])
    keep = torch.ones(c.M, dtype=torch.bool)
    keep[gone] = False
    x, a, b, scale, base, dout, u, dx = c.dev("x", "a", "b", "scale", "base", "dout", "u", "dx")
    rd = rows.to(torch.int32).cuda()
    out, kept = moe.lora(x, a, b, c.offsets, rows=rd, scale=scale, base=base, out=base.clone(), u=True)
    want, want_u = moe.lora(x, a, b, c.offsets, rows=c.rows_d, scale=scale, base=base, out=base.clone(), u=True)
    assert torch.equal(out[c.rows[keep]], want[c.rows[keep]])
    assert torch.equal(out[c.rows[gone]], base[c.rows[gone]])
    assert torch.equal(kept[keep], want_u[keep]) and not kept[gone].any()
    got = moe.lora_bwd(dout, x, u, a, b, c.offsets, rows=rd, scale=scale, base=dx, dx=dx.clone())
    dout0, u0 = dout.clone(), u.clone()
    dout0[c.rows[gone]] = 0
    want = moe.lora_bwd(dout0, x, u0, a, b, c.offsets, rows=c.rows_d, scale=scale, base=dx)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_no_rows():
    a, b = torch.ones((3, 64, 8), device="cuda"), torch.ones((3, 8, 32), device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, d, u = torch.empty((0, 64), device="cuda"), torch.empty((0, 32), device="cuda"), torch.empty((0, 8), device="cuda")
    assert moe.lora(x, a, b, off).shape == (0, 32)
    dx, da, db = moe.lora_bwd(d, x, u, a, b, off)
    assert dx.shape == (0, 64) and not da.any() and not db.any()
    # tokens, but none listed
    x, rows = torch.ones((5, 64), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert not moe.lora(x, a, b, off, rows=rows).any()


def test_gradients_against_differences():
    """All three gradients are the central differences of sum(dout * out) in 64 bits."""
    c = Case([3, 2], 5, 4, 2, "f32", 7, idle=1)
    dout, x, a, b, scale = c.dev("dout", "x", "a", "b", "scale")
    _, u = moe.lora(x, a, b, c.offsets, rows=c.rows_d, scale=scale, u=True)
    got = moe.lora_bwd(dout, x, torch.nan_to_num(u), a, b, c.offsets, rows=c.rows_d, scale=scale)
    v = {"x": c.x.double(), "a": c.a.double(), "b": c.b.double()}

    def total():
        return sum((f * (v["x"][t] @ v["a"][e]) @ v["b"][e] * c.dout[t].double()).sum().item() for e, _, t, f in c.segs())

    for name, g in zip("xab", got):
        flat, g = v[name].reshape(-1), g.cpu().double().reshape(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + 1e-4
            up = total()
            flat[i] = keep - 1e-4
            down = total()
            flat[i] = keep
            # linear in each value: the difference is exact but for 1e-12, the gradient's sums are fp32
            assert abs((up - down) / 2e-4 - g[i].item()) < 1e-4, name


def test_bad_arguments():
    x = torch.zeros((4, 64), device="cuda")
    a, b = torch.zeros((2, 64, 8), device="cuda"), torch.zeros((2, 8, 32), device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: moe.lora(x[:, :32].contiguous(), a, b, off), lambda: moe.lora(x, a, b[:, :4], off),
                 lambda: moe.lora(x, a, b, off[:2]), lambda: moe.lora(x, a, b, off.long()),
                 lambda: moe.lora(x, a, b, off, scale=off.float()), lambda: moe.lora(x, a.bfloat16(), b, off),
                 lambda: moe.lora(x, a, b, off, base=x), lambda: moe.lora(x.t().contiguous().t(), a, b, off),
                 lambda: moe.lora_bwd(x, x, None, a, b, off),
                 lambda: moe.lora_bwd(x[:, :32].contiguous(), x, x, a, b, off)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(moe.MoeError):
        moe.lora(x, torch.zeros((2, 64, 129), device="cuda"), torch.zeros((2, 129, 32), device="cuda"), off)
    with pytest.raises(moe.MoeError):
        moe.lora_bwd(x[:, :32].contiguous(), x, None, a, b, off)  # db needs u
