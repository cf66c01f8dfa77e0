"""The norms around a block and their gradients against plain fp64 computations (CPU,
torch double).

Tolerances, element by element, with S = 2^-23 (one binary32 step). A row's sums
pass through at most 64 additions in a lane, 6 between lanes and 16 between waves, so
any of them is off by 96 S of its terms' magnitudes. With m the mean and d = x - m:
m is off by 96 S mean|x|, d by that and S |d|, 1/sqrt(mean d^2 + eps) by (96 + 8) S and
what m's error does to it, relative; n = d rstd by the sum of these. Products and
additions after that add S each. Sums over tokens are off by (tokens + 32) S of their
terms' magnitudes and by the terms' own errors. The backward bounds send these through
the formulas, every absolute value taken. A result is off by half a step of its type
(bf16 2^-8, fp32 2^-24) on top."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe
from test_gpu_ffn import DT, STEP, check, half_step

pytestmark = pytest.mark.gpu

K96 = 104 * STEP


def unit(x, layer, eps):
    """n, its bound, 1/size."""
    m = x.mean(1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    e_m = K96 * x.abs().mean(1, keepdim=True) if layer else 0.0 * m
    d = x - m
    rstd = 1 / (d.square().mean(1, keepdim=True) + eps).sqrt()
    e_d = e_m + STEP * d.abs()
    rel = K96 + rstd ** 2 * (d.abs() * e_d).mean(1, keepdim=True)
    n = d * rstd
    return n, n.abs() * (rel + STEP) + e_d * rstd, rstd, rel


def unit_grad(e, ee, n, en, rstd, rel, layer):
    """Gradient of x from e, that of n, and its bound (ee, en: bounds of e and n)."""
    m1, a1 = (e * n).mean(1, keepdim=True), (e * n).abs().mean(1, keepdim=True)
    em1 = K96 * a1 + (ee * n.abs() + e.abs() * en + ee * en).mean(1, keepdim=True)
    m0 = e.mean(1, keepdim=True) if layer else 0.0 * m1
    em0 = K96 * e.abs().mean(1, keepdim=True) + ee.mean(1, keepdim=True) if layer else 0.0 * m1
    g = rstd * (e - n * m1 - m0)
    size = e.abs() + n.abs() * m1.abs() + m0.abs()
    eg = rstd * (ee + en * m1.abs() + n.abs() * em1 + en * em1 + em0 + size * (rel + 4 * STEP))
    return g, eg


class Case:
    def __init__(self, T, N, dt, res, kind, gate, post, pre, wt, seed, alpha=0.75, beta=0.5, eps=1e-5, mean=0.0,
                 residual=True):
        gen = torch.Generator().manual_seed(seed)
        self.T, self.N, self.dt, self.res = T, N, DT[dt], DT[res]
        self.layer, self.post, self.pre = kind == "layer", post, pre
        mk = lambda *s, sc=1.0, m=0.0, t=dt: (torch.randn(s, generator=gen) * sc + m).to(DT[t])  # noqa: E731
        self.z, self.r = mk(T, N, sc=0.7, m=mean), mk(T, N, sc=2.0, m=mean, t=res) if residual else None
        self.w = {}
        for side, there in (("post", post), ("pre", pre)):
            self.w["w_" + side] = mk(N, sc=0.2, m=1.0, t=wt) if there else None
            self.w["b_" + side] = mk(N, sc=0.3, t=wt) if there and self.layer else None
        shape = {"none": None, "channel": (N,), "token": (T, 1)}[gate]
        self.w["gate"] = mk(*shape, sc=0.5, m=0.5, t=wt) if shape else None
        self.mode, self.wt = gate, DT[wt]
        self.dh, self.dro = mk(T, N) if pre else None, mk(T, N, t=res)
        self.how = dict(alpha=alpha, beta=beta, eps=eps, kind=moe.NORM_LAYER if self.layer else moe.NORM_RMS, post=post)

    def dev(self, *names):
        get = lambda k: self.w[k] if k in self.w else getattr(self, k)  # noqa: E731
        return [get(k).cuda() if get(k) is not None else None for k in names]

    def weight(self, k):
        v = self.w[k]
        return v.double() if v is not None else torch.tensor(0.0 if k[0] == "b" else 1.0, dtype=torch.float64)

    def forward(self):
        z, r, w_post, b_post, gate, w_pre, b_pre = self.dev("z", "r", "w_post", "b_post", "gate", "w_pre", "b_pre")
        return moe.block_norm(z, r, w_post, b_post, gate, w_pre, b_pre, pre=self.pre, **self.how)

    def check_forward(self):
        ro, h = self.forward()
        alpha, beta, eps = (self.how[k] for k in ("alpha", "beta", "eps"))
        z = self.z.double()
        n, en = (unit(z, self.layer, eps)[:2]) if self.post else (z, 0.0 * z)
        w, b, g = self.weight("w_post"), self.weight("b_post"), self.weight("gate")
        u = n * w + b
        size = (n * w).abs() + b.abs()
        want = beta * g * u
        bound = beta * g.abs() * (en * w.abs() + 4 * STEP * size)
        if self.r is not None:
            want = want + alpha * self.r.double()
            bound = bound + STEP * (alpha * self.r.double()).abs() + STEP * want.abs()
        hs = half_step(self.res)
        check(ro, want, bound + hs * (want.abs() + bound), "r_out")
        assert (h is None) == (not self.pre)
        if not self.pre:
            return
        # h is the norm of r_out as stored
        n, en = unit(ro.cpu().double(), self.layer, eps)[:2]
        w, b = self.weight("w_pre"), self.weight("b_pre")
        want = n * w + b
        bound = en * w.abs() + 4 * STEP * ((n * w).abs() + b.abs())
        check(h, want, bound + half_step(self.dt) * (want.abs() + bound), "h")

    def backward(self, **kw):
        dh, dro, z, r, w_post, b_post, gate, w_pre = self.dev("dh", "dro", "z", "r", "w_post", "b_post", "gate", "w_pre")
        return moe.block_norm_bwd(dh, dro, z, r, w_post, b_post, gate, w_pre, **self.how, **kw)

    def check_backward(self, dw="f32", **kw):
        got = self.backward(dw_dtype=DT[dw], **kw)
        alpha, beta, eps = (self.how[k] for k in ("alpha", "beta", "eps"))
        tok = (self.T + 32) * STEP
        hw = half_step(DT[dw])

        def column(name, terms, err):
            want = terms.sum(0)
            b = tok * terms.abs().sum(0) + err.sum(0)
            check(got.pop(name), want, b + hw * (want.abs() + b), name)

        D, eD = self.dro.double(), 0.0 * self.dro.double()
        if self.pre:
            dh = self.dh.double()
            n, en, rstd, rel = unit(self.r.double(), self.layer, eps)
            e = dh * self.weight("w_pre")
            g, eg = unit_grad(e, STEP * e.abs(), n, en, rstd, rel, self.layer)
            D, eD = D + g, eg + STEP * (D + g).abs() + STEP * g.abs()
            column("dw_pre", dh * n, dh.abs() * en + STEP * (dh * n).abs())
            if self.layer:
                column("db_pre", dh, 0.0 * dh)
        hr = half_step(self.res)
        b = abs(alpha) * eD + STEP * (alpha * D).abs()
        check(got.pop("dr"), alpha * D, b + hr * ((alpha * D).abs() + b), "dr")
        z, gate = self.z.double(), self.weight("gate")
        if self.post:
            n, en, rstd, rel = unit(z, self.layer, eps)
        else:
            n, en = z, 0.0 * z
        w, bias = self.weight("w_post"), self.weight("b_post")
        br, ebr = beta * D, abs(beta) * eD + STEP * (beta * D).abs()
        u, eu = n * w + bias, en * w.abs() + 2 * STEP * ((n * w).abs() + bias.abs())
        if self.mode != "none":
            terms, err = br * u, ebr * u.abs() + br.abs() * eu + ebr * eu + 4 * STEP * (br * u).abs()
            if self.mode == "channel":
                # the kernel adds D n and D and multiplies by the weights after: the
                # terms' two parts are off separately
                err = err + tok * br.abs() * ((n * w).abs() + bias.abs())
                column("dgate", terms, err)
            else:
                want = terms.sum(1, keepdim=True)
                bb = K96 * (br.abs() * ((n * w).abs() + bias.abs())).sum(1, keepdim=True) + err.sum(1, keepdim=True)
                check(got.pop("dgate"), want, bb + hw * (want.abs() + bb), "dgate")
        du, edu = br * gate, (ebr + 2 * STEP * br.abs()) * gate.abs()
        if self.post:
            column("dw_post", du * n, edu * n.abs() + du.abs() * en + edu * en + 2 * STEP * (du * n).abs())
            if self.layer:
                column("db_post", du, edu)
            e = du * w
            du, edu = unit_grad(e, edu * w.abs() + STEP * e.abs(), n, en, rstd, rel, self.layer)
        check(got.pop("dz"), du, edu + half_step(self.dt) * (du.abs() + edu), "dz")
        assert not got


CASES = [
    # T, N, type, residual's, kind, gate, post, pre, weights'
    (1, 1, "f32", "f32", "rms", "none", True, True, "f32"), (1, 4096, "bf16", "bf16", "rms", "none", True, True, "bf16"),
    (3, 7, "f32", "f32", "layer", "channel", True, True, "f32"), (1, 129, "bf16", "f32", "layer", "token", True, True, "bf16"),
    (5, 512, "bf16", "bf16", "layer", "channel", True, True, "f32"), (37, 513, "bf16", "f32", "rms", "channel", True, True, "f32"),
    (777, 1501, "bf16", "bf16", "layer", "channel", True, True, "bf16"), (2049, 100, "f32", "f32", "rms", "token", True, True, "bf16"),
    (2500, 1000, "bf16", "f32", "layer", "none", True, True, "f32"), (2100, 2047, "bf16", "bf16", "rms", "channel", True, False, "bf16"),
    (2048, 4096, "bf16", "bf16", "rms", "token", False, True, "f32"), (64, 2048, "bf16", "bf16", "rms", "none", False, False, "bf16"),
    (600, 4104, "bf16", "f32", "rms", "channel", True, True, "f32"), (33, 8192, "f32", "f32", "layer", "token", True, True, "f32"),
    (520, 9001, "bf16", "bf16", "rms", "none", True, True, "bf16"), (17, 16384, "bf16", "f32", "layer", "channel", True, True, "f32"),
    (5, 20000, "bf16", "bf16", "layer", "token", True, True, "bf16"), (3, 65535, "f32", "f32", "rms", "channel", True, True, "f32"),
    (520, 17000, "bf16", "bf16", "rms", "none", True, False, "bf16"), (2, 40000, "bf16", "f32", "layer", "none", False, True, "f32"),
]


@pytest.mark.parametrize("T,N,dt,res,kind,gate,post,pre,wt", CASES)
def test_forward(T, N, dt, res, kind, gate, post, pre, wt):
    Case(T, N, dt, res, kind, gate, post, pre, wt, T + N).check_forward()


@pytest.mark.parametrize("T,N,dt,res,kind,gate,post,pre,wt", CASES)
def test_backward(T, N, dt, res, kind, gate, post, pre, wt):
    Case(T, N, dt, res, kind, gate, post, pre, wt, T + N + 1).check_backward(dw=wt)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_large_means_and_rows_of_zeros(kind):
    c = Case(70, 600, "f32", "f32", kind, "none", True, True, "f32", 3, mean=300.0)
    c.z[5], c.r[7], c.z[9], c.r[9] = 0, 0, 0, 0
    c.check_forward()
    c.check_backward()


def test_without_a_residual_stream():
    Case(130, 640, "bf16", "bf16", "rms", "channel", True, True, "bf16", 4, residual=False).check_forward()


@pytest.mark.parametrize("dt,res,N", [("bf16", "f32", 1000), ("f32", "f32", 333), ("bf16", "bf16", 4096)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_alone(dt, res, N, kind):
    """z None: h is the norm of r, dr its gradient."""
    c = Case(45, N, dt, res, kind, "none", False, True, dt, 5)
    c.how["post"] = False
    r, w, b, dh, dro = c.dev("r", "w_pre", "b_pre", "dh", "dro")
    none, h = moe.block_norm(None, r, w_pre=w, b_pre=b, eps=1e-5, kind=c.how["kind"], h=torch.empty((45, N), dtype=c.dt, device="cuda"))
    assert none is None
    n, en, rstd, rel = unit(c.r.double(), c.layer, 1e-5)
    w64, b64 = c.weight("w_pre"), c.weight("b_pre")
    want, bound = n * w64 + b64, en * w64.abs() + 4 * STEP * ((n * w64).abs() + b64.abs())
    check(h, want, bound + half_step(c.dt) * (want.abs() + bound), "h")
    for extra in (None, dro):
        got = moe.block_norm_bwd(dh, extra, None, r, w_pre=w, eps=1e-5, kind=c.how["kind"], alpha=3.0, dw_dtype=torch.float32)
        e = c.dh.double() * w64
        g, eg = unit_grad(e, STEP * e.abs(), n, en, rstd, rel, c.layer)
        if extra is not None:
            g = g + c.dro.double()
        eg = eg + 2 * STEP * (g.abs() + c.dro.double().abs())
        check(got.pop("dr"), g, eg + half_step(c.res) * (g.abs() + eg), "dr")
        terms = c.dh.double() * n
        b = (45 + 32) * STEP * terms.abs().sum(0) + (c.dh.double().abs() * en).sum(0)
        check(got.pop("dw_pre"), terms.sum(0), b + 2.0 ** -24 * terms.sum(0).abs(), "dw_pre")
        if c.layer:
            s = c.dh.double()
            check(got.pop("db_pre"), s.sum(0), (45 + 32) * STEP * s.abs().sum(0) + 2.0 ** -24 * s.sum(0).abs(), "db_pre")
        assert not got


def test_in_place_and_partial_outputs():
    c = Case(300, 1024, "bf16", "f32", "rms", "channel", True, True, "f32", 6)
    ro, h = c.forward()
    z, r, w_post, gate, w_pre = c.dev("z", "r", "w_post", "gate", "w_pre")
    ro2, h2 = moe.block_norm(z, r, w_post, None, gate, w_pre, r_out=r, **c.how)
    assert ro2 is r and torch.equal(ro2, ro) and torch.equal(h2, h)
    full = c.backward()
    assert set(c.backward(need_dw=False)) == {"dr", "dz"}
    for key, kw in (("dr", dict(need_dr=False)), ("dz", dict(need_dz=False))):
        part = c.backward(**kw)
        assert key not in part and all(torch.equal(part[k], full[k]) for k in part)


def test_no_rows():
    z = torch.empty((0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    ro, h = moe.block_norm(z, z, w, w_pre=w)
    assert ro.shape == h.shape == (0, 64)
    got = moe.block_norm_bwd(z, z, z, z, w, gate=w, w_pre=w)
    for k in ("dw_post", "dw_pre", "dgate"):
        assert got[k].tolist() == [0.0] * 64


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradient_against_differences(kind):
    """Every gradient is the central difference of sum(dh * h + dr_out * r_out) in 64
    bits: its error is of order h^2, 1e-10, against the fp32 gradients' 1e-5."""
    c = Case(3, 6, "f32", "f32", kind, "channel", True, True, "f32", 7)
    layer, eps = c.layer, 1e-5
    v = {k: t.double() for k, t in (("z", c.z), ("r", c.r), *((k, t) for k, t in c.w.items() if t is not None))}
    ro, _ = c.forward()
    one = lambda x: unit(x, layer, eps)[0]  # noqa: E731

    def out(v):
        u = one(v["z"]) * v["w_post"] + v.get("b_post", 0.0)
        r = 0.75 * v["r"] + 0.5 * v["gate"] * u
        return r, one(r) * v["w_pre"] + v.get("b_pre", 0.0)

    def total(v):
        r, h = out(v)
        return ((c.dh.double() * h).sum() + (c.dro.double() * r).sum()).item()

    dh, dro, z, w_post, b_post, gate, w_pre = c.dev("dh", "dro", "z", "w_post", "b_post", "gate", "w_pre")
    got = moe.block_norm_bwd(dh, dro, z, ro, w_post, b_post, gate, w_pre, **c.how)
    for name, t in v.items():
        g = got["d" + name].cpu().double().reshape(-1)
        flat = t.reshape(-1)
        for i in range(flat.numel()):
            keep, step = flat[i].item(), 1e-5
            flat[i] = keep + step
            up = total(v)
            flat[i] = keep - step
            down = total(v)
            flat[i] = keep
            assert abs((up - down) / (2 * step) - g[i].item()) < 2e-4, name


def test_bad_arguments():
    z = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        moe.block_norm(z, z[:3])
    with pytest.raises(ValueError):
        moe.block_norm(z, z, w[:32])
    with pytest.raises(ValueError):
        moe.block_norm(z, z, w, w_pre=w.bfloat16())
    with pytest.raises(ValueError):
        moe.block_norm(z, z, gate=w[:5])
    with pytest.raises(ValueError):
        moe.block_norm(z, z.t().contiguous().t())
    with pytest.raises(moe.MoeError):
        moe.block_norm(z, z, w, b_post=w)  # an RMS norm has no bias
    with pytest.raises(moe.MoeError):
        moe.block_norm(z, z.bfloat16(), w)
    with pytest.raises(moe.MoeError):
        moe.block_norm_bwd(None, None, z, z, w)
