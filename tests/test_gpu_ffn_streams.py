"""Calls that run on another stream than the caller's current one."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe

pytestmark = pytest.mark.gpu


def operands():
    gen = torch.Generator().manual_seed(0)
    mk = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    A, H, N, e = 700, 512, 256, 4
    off = torch.tensor([0, 300, 300, 650, 700], dtype=torch.int32, device="cuda")
    x, wg, wu, d, g, u = mk(A, H), mk(e, H, N), mk(e, H, N), mk(A, N), mk(A, N), mk(A, N)
    q, scale = moe.quant_mxfp4_weights(wg)
    torch.cuda.synchronize()
    return {
        "gmm_glu": lambda **k: moe.gmm_glu(x, wg, wu, off, save=True, **k),
        "gmm_glu_bwd": lambda **k: moe.gmm_glu_bwd(d, g, u, x, wg, wu, off, **k),
        "gmm_dgrad": lambda **k: (moe.gmm_dgrad(d, wg, off, **k),),
        "gmm_wgrad": lambda **k: (moe.gmm_wgrad(x, d, off, **k),),
        "quant_mxfp4_rows": lambda **k: moe.quant_mxfp4_rows(x, values=True, **k),
        "quant_mxfp4_weights": lambda **k: moe.quant_mxfp4_weights(wg, values=True, **k),
        "gmm_mxfp4_dyn": lambda **k: (moe.gmm_mxfp4_dyn(x, q, scale, off, **k),),
    }


OPS = ("gmm_glu", "gmm_glu_bwd", "gmm_dgrad", "gmm_wgrad", "quant_mxfp4_rows", "quant_mxfp4_weights", "gmm_mxfp4_dyn")


def keep_busy(stream):
    """A few milliseconds of products on `stream`."""
    a = torch.ones((8192, 8192), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(3):
            b = a @ a
    return a, b


@pytest.mark.parametrize("op", OPS)
def test_results_of_another_stream_may_be_read_at_once(op):
    """Tensors that a call allocates are ordered with the caller's stream, though
    `stream` has work before it."""
    call = operands()[op]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # later blocks of the stream's memory hold other values
        junk = [torch.full_like(t, 1) for t in want]
    torch.cuda.synchronize()
    del junk
    hold = keep_busy(side)
    got = [t.clone() for t in call(stream=side)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del hold


def test_results_of_another_stream_may_be_dropped_at_once():
    """Memory of a dropped result is not given to its stream's next call while the
    caller's stream still reads it."""
    call = operands()["gmm_dgrad"]
    want = call()[0].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r = call(stream=side)[0]
    hold = keep_busy(torch.cuda.current_stream())
    got = r.clone()  # runs after the products
    del r
    with torch.cuda.stream(side):
        junk = [torch.full_like(want, 1) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del hold, junk


def test_given_outputs_leave_the_streams_apart():
    """With every output given the caller's stream does not wait."""
    call = operands()["gmm_dgrad"]
    out = torch.empty_like(call()[0])
    side = torch.cuda.Stream()
    hold = keep_busy(side)
    call(stream=side, out=out)
    mark = torch.cuda.Event()
    mark.record()
    mark.synchronize()
    assert not side.query()  # the products are still running
    torch.cuda.synchronize()
    del hold


def test_forked_stream_inside_a_captured_graph():
    """A call on a stream forked from the capturing one: its results are joined to
    the capture, and replays read them behind it."""
    call = operands()["gmm_glu_bwd"]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        parts = call(stream=side)
        got = [t + 0 for t in parts]
        del parts
    for _ in range(3):
        for t in got:
            t.fill_(7.0)
        again = call()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, again):
            assert torch.equal(a, b) and torch.equal(c, b)
