"""Refusals of the gated feed-forward and the grouped GEMM's gradients, without
a GPU: every case carries at least one invalid argument (or no work), so
nothing is enqueued."""
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


def glu(a=P, a_rows=50, src=None, div=1, dt=moe.BF16, wg=P, wu=P, ldw=64, off=P, e=8, A=100, Hin=128, N=64,
        act=moe.ACT_SILU, out=P, gate=None, up=None):
    return L.moe_gmm_glu(a, a_rows, src, div, dt, wg, wu, ldw, off, e, A, Hin, N, act, out, gate, up, None)


SHAPES = [
    (dict(dt=moe.FP8_E4M3), moe.ERR_BAD_DTYPE), (dict(dt=9), moe.ERR_BAD_DTYPE),
    (dict(e=0), moe.ERR_BAD_SHAPE), (dict(e=257), moe.ERR_BAD_SHAPE),
    (dict(A=-1), moe.ERR_BAD_SHAPE), (dict(A=52428800), moe.ERR_BAD_SHAPE),
    (dict(Hin=0), moe.ERR_BAD_SHAPE), (dict(Hin=65536), moe.ERR_BAD_SHAPE),
    (dict(N=0, ldw=64), moe.ERR_BAD_SHAPE), (dict(N=65536, ldw=65536), moe.ERR_BAD_SHAPE),
]
GATHER = [
    (dict(src=P, div=0), moe.ERR_BAD_SHAPE), (dict(src=P, a_rows=0), moe.ERR_BAD_SHAPE),
    (dict(src=P, a_rows=-1), moe.ERR_BAD_SHAPE), (dict(src=MIS), moe.ERR_MISALIGNED),
    (dict(src=P, a_rows=1 << 23), moe.ERR_UNSUPPORTED),
    (dict(src=P, a_rows=1 << 22, dt=moe.F32), moe.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", SHAPES + GATHER + [
    (dict(ldw=63), moe.ERR_BAD_SHAPE), (dict(ldw=131072), moe.ERR_BAD_SHAPE),
    (dict(act=4), moe.ERR_UNSUPPORTED), (dict(act=-1), moe.ERR_UNSUPPORTED),
    (dict(a=None), moe.ERR_NULL_POINTER), (dict(wg=None), moe.ERR_NULL_POINTER),
    (dict(wu=None), moe.ERR_NULL_POINTER), (dict(off=None), moe.ERR_NULL_POINTER),
    (dict(out=None), moe.ERR_NULL_POINTER), (dict(gate=P), moe.ERR_NULL_POINTER),
    (dict(up=P), moe.ERR_NULL_POINTER),
    (dict(a=MIS), moe.ERR_MISALIGNED), (dict(wg=MIS), moe.ERR_MISALIGNED), (dict(wu=MIS), moe.ERR_MISALIGNED),
    (dict(off=MIS), moe.ERR_MISALIGNED), (dict(out=MIS), moe.ERR_MISALIGNED),
    (dict(gate=MIS, up=P), moe.ERR_MISALIGNED), (dict(gate=P, up=MIS), moe.ERR_MISALIGNED),
])
def test_glu_validation(kw, status):
    assert glu(**kw) == status


def test_glu_no_rows_is_noop():
    assert glu(A=0, a=None, wg=None, wu=None, off=None, out=None) == moe.OK


def glu_bwd(d=P, g=P, u=P, a=P, a_rows=50, src=None, div=1, dt=moe.BF16, wg=P, wu=P, ldw=64, off=P, e=8, A=100,
            Hin=128, N=64, act=moe.ACT_SILU, da=P, dwg=P, dwu=P, lddw=None, ws=P, ws_bytes=1 << 20):
    return L.moe_gmm_glu_bwd(d, g, u, a, a_rows, src, div, dt, wg, wu, ldw, off, e, A, Hin, N, act, da, dwg, dwu,
                             N if lddw is None else lddw, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", SHAPES + GATHER + [
    (dict(ldw=63), moe.ERR_BAD_SHAPE), (dict(lddw=63), moe.ERR_BAD_SHAPE), (dict(lddw=131072), moe.ERR_BAD_SHAPE),
    (dict(act=4), moe.ERR_UNSUPPORTED),
    (dict(d=None), moe.ERR_NULL_POINTER), (dict(g=None), moe.ERR_NULL_POINTER), (dict(u=None), moe.ERR_NULL_POINTER),
    (dict(a=None), moe.ERR_NULL_POINTER), (dict(wg=None), moe.ERR_NULL_POINTER),
    (dict(wu=None), moe.ERR_NULL_POINTER), (dict(off=None), moe.ERR_NULL_POINTER),
    (dict(dwg=None), moe.ERR_NULL_POINTER), (dict(dwu=None), moe.ERR_NULL_POINTER),
    (dict(da=None, dwg=None, dwu=None), moe.ERR_NULL_POINTER), (dict(ws=None), moe.ERR_NULL_POINTER),
    (dict(ws_bytes=2 * 100 * 64 * 2 - 1), moe.ERR_WORKSPACE_TOO_SMALL),
] + [(dict([(k, MIS)]), moe.ERR_MISALIGNED) for k in
     ("d", "g", "u", "a", "wg", "wu", "off", "da", "dwg", "dwu", "ws")])
def test_glu_bwd_validation(kw, status):
    assert glu_bwd(**kw) == status


def test_glu_bwd_workspace_size():
    assert moe.gmm_glu_bwd_workspace_size(moe.BF16, 8, 100, 128, 64) == 2 * 100 * 64 * 2
    assert moe.gmm_glu_bwd_workspace_size(moe.F32, 8, 0, 128, 64) == 0
    # above 4 GiB
    assert moe.gmm_glu_bwd_workspace_size(moe.F32, 8, 1 << 20, 128, 4096) == 2 << 34
    for bad in ((moe.FP8_E4M3, 8, 1, 1, 1), (moe.BF16, 0, 1, 1, 1), (moe.BF16, 8, 1, 0, 1), (moe.BF16, 8, -1, 1, 1)):
        with pytest.raises(moe.MoeError):
            moe.gmm_glu_bwd_workspace_size(*bad)


def test_glu_bwd_no_rows_without_weight_gradients_is_noop():
    assert glu_bwd(A=0, d=None, g=None, u=None, a=None, wg=None, wu=None, dwg=None, dwu=None, ws=None,
                   ws_bytes=0) == moe.OK


def dgrad(d=P, dt=moe.BF16, w=P, off=P, e=8, A=100, Hin=128, N=64, da=P, ldw=None):
    return L.moe_gmm_dgrad(d, dt, w, off, e, A, Hin, N, da, None)


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict([(k, None)]), moe.ERR_NULL_POINTER) for k in ("d", "w", "off", "da")] + [
    (dict([(k, MIS)]), moe.ERR_MISALIGNED) for k in ("d", "w", "off", "da")])
def test_dgrad_validation(kw, status):
    assert dgrad(**kw) == status


def test_dgrad_no_rows_is_noop():
    assert dgrad(A=0, d=None, w=None, off=None, da=None) == moe.OK


def wgrad(a=P, a_rows=50, src=None, div=1, d=P, dt=moe.BF16, off=P, e=8, A=100, Hin=128, N=64, dw=P, dwdt=None,
          ldw=None, ws=None, ws_bytes=0):
    return L.moe_gmm_wgrad(a, a_rows, src, div, d, dt, off, e, A, Hin, N, dw, dt if dwdt is None else dwdt, ws,
                           ws_bytes, None)


@pytest.mark.parametrize("kw,status", SHAPES + GATHER + [
    (dict(dt=moe.F32, dwdt=moe.BF16), moe.ERR_BAD_DTYPE), (dict(dwdt=moe.FP8_E4M3), moe.ERR_BAD_DTYPE)] + [
    (dict([(k, None)]), moe.ERR_NULL_POINTER) for k in ("a", "d", "off", "dw")] + [
    (dict([(k, MIS)]), moe.ERR_MISALIGNED) for k in ("a", "d", "off", "dw")])
def test_wgrad_validation(kw, status):
    assert wgrad(**kw) == status


def test_wgrad_workspace():
    # enough tiles: none; a dense FFN's few: the partial sums of 2 or more parts
    assert moe.gmm_wgrad_workspace_size(moe.BF16, 64, 98304, 2048, 1408) == 0
    need = moe.gmm_wgrad_workspace_size(moe.BF16, 1, 32768, 1024, 512)
    assert need >= 2 * 1024 * 512 * 4 and need % (1024 * 512 * 4) == 0
    kw = dict(e=1, A=32768, Hin=1024, N=512)
    assert wgrad(**kw) == moe.ERR_NULL_POINTER
    assert wgrad(ws=P, ws_bytes=need - 1, **kw) == moe.ERR_WORKSPACE_TOO_SMALL
    assert wgrad(ws=MIS, ws_bytes=need, **kw) == moe.ERR_MISALIGNED
    assert moe.gmm_glu_bwd_workspace_size(moe.BF16, 1, 32768, 1024, 512) > 32768 * 2 * 512 * 2
    for bad in ((moe.FP8_E4M3, 8, 1, 1, 1), (moe.BF16, 0, 1, 1, 1), (moe.BF16, 8, 1, 0, 1), (moe.BF16, 8, -1, 1, 1)):
        with pytest.raises(moe.MoeError):
            moe.gmm_wgrad_workspace_size(*bad)


def test_silu_and_gelu_belong_to_the_gated_block():
    """The plain grouped GEMM and the layer refuse them as before."""
    for act in (moe.ACT_SILU, moe.ACT_GELU):
        assert L.moe_gmm(P, moe.BF16, 0, None, P, moe.BF16, 0, None, P, 8, 100, 128, 64, act, P, moe.BF16, P, 1 << 40,
                         None) == moe.ERR_UNSUPPORTED


def test_binding_refuses_host_tensors_and_mismatches():
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    w = torch.zeros((2, 8, 16), dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        moe.gmm_glu(x, w, w, off)
    with pytest.raises(ValueError, match="disagree"):
        moe.gmm_glu(x[:, :4], w, w, off)
    with pytest.raises(ValueError, match="disagree"):
        moe.gmm_glu(x.float(), w, w, off)
    with pytest.raises(ValueError, match="offsets"):
        moe.gmm_glu(x, w, w, off[:2])
    with pytest.raises(ValueError, match="offsets"):
        moe.gmm_glu(x, w, w, off.long())
    with pytest.raises(ValueError, match="rows"):
        moe.gmm_glu(x, w, w, off, rows=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="agree in shape"):
        moe.gmm_glu(x, w, w[:1], off)
    with pytest.raises(ValueError, match="contiguous"):
        moe.gmm_glu(x, w.transpose(1, 2).contiguous().transpose(1, 2), w, off)
    with pytest.raises(ValueError, match="strides"):
        moe.gmm_glu(x, w, torch.zeros((2, 8, 32), dtype=torch.bfloat16)[:, :, :16], off)
    with pytest.raises(TypeError):
        b = torch.zeros((2, 8, 16), dtype=torch.uint8)
        moe.gmm_glu(x.to(torch.uint8), b, b, off)
