"""Refusals of the MXFP4 quantisers and of the product that quantises its rows,
without a GPU: every case carries at least one invalid argument (or no work),
so nothing is enqueued."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe

P = 0x100000   # 16-byte aligned stand-in address, never dereferenced
MIS = 0x100004

L = None


@pytest.fixture(autouse=True)
def _lib():
    global L
    L = moe.lib()


def rows(x=P, dt=moe.BF16, x_rows=10, H=256, src=None, div=1, n=10, q=P, sc=P, values=P):
    return L.moe_quant_mxfp4_rows(x, dt, x_rows, H, src, div, n, q, sc, values, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=moe.FP8_E4M3), moe.ERR_BAD_DTYPE), (dict(H=0), moe.ERR_BAD_SHAPE), (dict(H=65536), moe.ERR_BAD_SHAPE),
    (dict(H=128), moe.ERR_UNSUPPORTED), (dict(H=300), moe.ERR_UNSUPPORTED), (dict(x_rows=-1), moe.ERR_BAD_SHAPE),
    (dict(n=-1), moe.ERR_BAD_SHAPE), (dict(n=11), moe.ERR_BAD_SHAPE), (dict(n=52428800, src=P), moe.ERR_BAD_SHAPE),
    (dict(src=P, div=0), moe.ERR_BAD_SHAPE), (dict(x=None), moe.ERR_NULL_POINTER),
    (dict(q=None), moe.ERR_NULL_POINTER), (dict(sc=None), moe.ERR_NULL_POINTER),
    (dict(q=None, sc=None, values=None), moe.ERR_NULL_POINTER),
    (dict(x=MIS), moe.ERR_MISALIGNED), (dict(src=MIS), moe.ERR_MISALIGNED), (dict(q=MIS), moe.ERR_MISALIGNED),
    (dict(sc=MIS), moe.ERR_MISALIGNED), (dict(values=MIS), moe.ERR_MISALIGNED),
])
def test_quant_rows_validation(kw, status):
    assert rows(**kw) == status


def test_quant_rows_no_rows_is_noop():
    assert rows(n=0, x=None, q=None, sc=None, values=None) == moe.OK


def weights(w=P, dt=moe.BF16, e=4, Hin=256, N=64, q=P, sc=P, values=P):
    return L.moe_quant_mxfp4_weights(w, dt, e, Hin, N, q, sc, values, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=moe.FP8_E4M3), moe.ERR_BAD_DTYPE), (dict(e=0), moe.ERR_BAD_SHAPE), (dict(e=257), moe.ERR_BAD_SHAPE),
    (dict(Hin=0), moe.ERR_BAD_SHAPE), (dict(N=65536), moe.ERR_BAD_SHAPE), (dict(Hin=128), moe.ERR_UNSUPPORTED),
    (dict(N=24), moe.ERR_UNSUPPORTED), (dict(w=None), moe.ERR_NULL_POINTER), (dict(q=None), moe.ERR_NULL_POINTER),
    (dict(sc=None), moe.ERR_NULL_POINTER), (dict(q=None, sc=None, values=None), moe.ERR_NULL_POINTER),
] + [(dict([(k, MIS)]), moe.ERR_MISALIGNED) for k in ("w", "q", "sc", "values")])
def test_quant_weights_validation(kw, status):
    assert weights(**kw) == status


def dyn(x=P, dt=moe.BF16, x_rows=100, src=None, div=1, w=P, sw=P, off=P, e=8, A=100, Hin=512, N=64, act=moe.ACT_NONE,
        out=P, ws=P, ws_bytes=1 << 30):
    return L.moe_gmm_mxfp4_dyn(x, dt, x_rows, src, div, w, sw, off, e, A, Hin, N, act, out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=moe.FP8_E4M3), moe.ERR_BAD_DTYPE), (dict(x_rows=99), moe.ERR_BAD_SHAPE),
    (dict(x_rows=-1), moe.ERR_BAD_SHAPE), (dict(src=P, div=0), moe.ERR_BAD_SHAPE), (dict(e=0), moe.ERR_BAD_SHAPE),
    (dict(e=257), moe.ERR_BAD_SHAPE), (dict(A=-1), moe.ERR_BAD_SHAPE),
    (dict(A=52428800, x_rows=52428800), moe.ERR_BAD_SHAPE), (dict(Hin=128), moe.ERR_UNSUPPORTED),
    (dict(N=24), moe.ERR_UNSUPPORTED), (dict(Hin=0), moe.ERR_BAD_SHAPE), (dict(N=65536), moe.ERR_BAD_SHAPE),
    (dict(act=moe.ACT_SILU), moe.ERR_UNSUPPORTED),
] + [(dict([(k, None)]), moe.ERR_NULL_POINTER) for k in ("x", "w", "sw", "off", "out")]
  + [(dict([(k, MIS)]), moe.ERR_MISALIGNED) for k in ("x", "src", "w", "sw", "off", "out")])
def test_dyn_validation(kw, status):
    assert dyn(**kw) == status


def test_dyn_workspace():
    big = dict(e=1, A=4096, x_rows=4096)
    need = moe.gmm_mxfp4_dyn_workspace_size(1, 4096, 512, 64)
    assert need >= 4096 * (512 // 2 + 512 // 32)
    assert dyn(ws=None, **big) == moe.ERR_NULL_POINTER
    assert dyn(ws=MIS, **big) == moe.ERR_MISALIGNED
    assert dyn(ws_bytes=need - 1, **big) == moe.ERR_WORKSPACE_TOO_SMALL
    for bad in ((0, 1, 256, 16), (1, -1, 256, 16), (1, 1, 128, 16), (1, 1, 256, 8)):
        with pytest.raises(moe.MoeError):
            moe.gmm_mxfp4_dyn_workspace_size(*bad)


def test_dyn_no_rows_is_noop():
    assert dyn(A=0, x=None, w=None, sw=None, off=None, out=None, ws=None, ws_bytes=0) == moe.OK


def test_binding_refuses_host_tensors_and_mismatches():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        moe.quant_mxfp4_rows(x)
    with pytest.raises(ValueError, match="GPU"):
        moe.quant_mxfp4_weights(torch.zeros((2, 256, 16)))
    with pytest.raises(TypeError):
        moe.quant_mxfp4_rows(x.to(torch.uint8))
    with pytest.raises(ValueError, match="disagree"):
        moe.gmm_mxfp4_dyn(x, torch.zeros((2, 64, 16), dtype=torch.uint8), x, x)
