"""Adapter calls whose row list names fewer rows than it has entries, and no output
given: the rows that nobody lists get base's values, or zeros."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe
from test_gpu_ffn import DT

pytestmark = pytest.mark.gpu


class Padded:
    """A list of M entries for T rows, as a program with one length for every step makes
    it: each adapter's rows, then rows of no adapter, then -1; entries outside the
    tensors between them too."""

    def __init__(self, counts, T, M, H, N, R, dt, seed, idle=2, gone=()):
        gen = torch.Generator().manual_seed(seed)
        mk = lambda *s: torch.randn(s, generator=gen).to(DT[dt]).cuda()  # noqa: E731
        n = sum(counts)
        rows = torch.full((M,), -1, dtype=torch.int32)
        rows[:n + idle] = torch.randperm(T, generator=gen)[:n + idle].to(torch.int32)
        for i, v in zip(range(0, n, 3), gone):
            rows[i] = v
        self.T, self.M, self.e = T, M, len(counts)
        self.offsets = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        self.rows = rows.cuda()
        listed = torch.zeros(T, dtype=torch.bool)
        listed[rows[(rows >= 0) & (rows < T)].long()] = True
        self.listed = listed.cuda()
        self.x, self.base, self.dout, self.dx = mk(T, H), mk(T, N), mk(T, N), mk(T, H)
        self.a, self.b = mk(self.e, H, R), mk(self.e, R, N)
        self.u = torch.randn((M, R), generator=gen).cuda()

    def forward(self, **kw):
        return moe.lora(self.x, self.a, self.b, self.offsets, rows=self.rows, **kw)

    def backward(self, **kw):
        return moe.lora_bwd(self.dout, self.x, self.u, self.a, self.b, self.offsets, rows=self.rows, **kw)


def soil(t):
    """Leaves t's sizes in the allocator's cache, full of a value that no result has."""
    for _ in range(3):
        junk = [torch.full_like(t, 12345.0) for _ in range(4)]
        del junk


CASES = [
    ([1], 5, 5, 64, 64, 4, "f32", dict(idle=0)), ([3, 0, 2], 64, 64, 136, 264, 16, "bf16", {}),
    ([30, 20], 100, 130, 257, 401, 5, "f32", dict(gone=[-1, 100, 2 ** 31 - 1, -2 ** 31])),
    ([500, 0, 100], 1501, 1600, 128, 1031, 8, "bf16", dict(gone=[1501])), ([0, 0], 70, 80, 64, 72, 8, "bf16", {}),
    ([0], 300, 300, 64, 40, 4, "f32", dict(idle=0)), ([2500, 700], 9000, 9000, 512, 1024, 64, "bf16", dict(idle=100)),
    ([600, 600], 1210, 1211, 2048, 64, 100, "bf16", {}), ([40], 43, 50, 4, 3, 2, "bf16", {}), ([9], 20, 14, 72, 64, 8, "f32", {}),
]


@pytest.mark.parametrize("counts,T,M,H,N,R,dt,more", CASES)
def test_rows_nobody_lists(counts, T, M, H, N, R, dt, more):
    c = Padded(counts, T, M, H, N, R, dt, T + N, **more)
    for base in (c.base, None):
        want = c.forward(base=base, out=base.clone() if base is not None else torch.zeros_like(c.base))
        soil(c.base)
        got = c.forward(base=base)
        rest = base if base is not None else torch.zeros_like(c.base)
        assert torch.equal(got[~c.listed], rest[~c.listed]) and torch.equal(got, want)
        soil(c.base)
        got, _ = c.forward(base=base, u=True)
        assert torch.equal(got, want)
    for base in (c.dx, None):
        want = c.backward(base=base, dx=base.clone() if base is not None else torch.zeros_like(c.dx))
        for need in (dict(), dict(need_da=False, need_db=False), dict(need_da=False)):
            soil(c.dx)
            got = c.backward(base=base, **need)
            rest = base if base is not None else torch.zeros_like(c.dx)
            assert torch.equal(got[0][~c.listed], rest[~c.listed])
            for g, w in zip(got, want):
                assert g is None or torch.equal(g, w)


def test_in_a_graph():
    """Captured once, the list changes between replays: every replay fills what its own
    list leaves out, whatever the last one left in the output and the workspace."""
    c = Padded([30, 20], 90, 96, 128, 264, 8, "bf16", 1)
    c.forward(base=c.base)
    c.backward(base=c.dx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.forward(base=c.base)
        dx, da, db = c.backward(base=c.dx)
    for i, (n, idle) in enumerate([(50, 0), (7, 20), (50, 40), (0, 5)]):
        rows = torch.full((96,), -1, dtype=torch.int32)
        rows[:n + idle] = torch.randperm(90, generator=torch.Generator().manual_seed(i))[:n + idle].to(torch.int32)
        c.rows.copy_(rows)
        c.offsets.copy_(torch.tensor([0, n // 2, n], dtype=torch.int32))
        want = [c.forward(base=c.base, out=c.base.clone()), *c.backward(base=c.dx, dx=c.dx.clone())]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, dx, da, db), want):
            assert torch.equal(a, b)


def test_given_outputs_are_left_alone():
    """With `out` given, rows that nobody lists stay as they are there."""
    c = Padded([30, 20], 90, 96, 64, 72, 8, "f32", 2)
    out, dx = torch.full_like(c.base, 3.0), torch.full_like(c.dx, 4.0)
    c.forward(base=c.base, out=out)
    c.backward(base=c.dx, dx=dx)
    assert (out[~c.listed] == 3).all() and (dx[~c.listed] == 4).all()
