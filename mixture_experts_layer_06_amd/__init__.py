"""Python binding of the gfx950 MoE C-ABI library (libmoe.so).

Argument marshalling only: every step of the layer runs in the HIP kernels
behind include/moe.h. torch supplies device memory (tensors) and the stream
(torch.cuda.current_stream()). There is no CPU fallback: if libmoe.so is
missing the import of any entry point raises.

Tensor element types: torch.float32 -> MOE_F32, torch.bfloat16 -> MOE_BF16,
torch.uint8 or torch.float8_e4m3fn -> MOE_FP8_E4M3 (OCP E4M3 bytes).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch  # noqa: F401  (loads the HIP runtime libmoe.so binds to)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

# moe.h enums
OK, ERR_NULL_POINTER, ERR_BAD_SHAPE, ERR_BAD_DTYPE, ERR_UNSUPPORTED = 0, 1, 2, 3, 4
ERR_WORKSPACE_TOO_SMALL, ERR_MISALIGNED, ERR_DEVICE, ERR_SCRATCH_LIMIT = 5, 6, 7, 8
NOALLOC_SCRATCH_BYTES = 32 << 20  # MOE_NOALLOC_SCRATCH_BYTES
F32, BF16, FP8_E4M3 = 0, 1, 2
QUANT_NONE, QUANT_PER_TENSOR, QUANT_PER_TOKEN = 0, 1, 3
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3

EXPORTS = ("moe_status_string", "moe_version", "moe_route_workspace_size", "moe_route",
           "moe_permute_workspace_size", "moe_permute", "moe_gmm_workspace_size", "moe_gmm",
           "moe_gmm_gather", "moe_gmm_scatter", "moe_gmm_routed_shared", "moe_gmm_mx_routed_shared", "moe_gmm_mx", "moe_gmm_mxfp4", "moe_combine", "moe_sum_slots",
           "moe_quant_rows", "moe_layer_workspace_size", "moe_layer", "moe_layer_fp8_workspace_size",
           "moe_layer_fp8", "moe_layer_noalloc", "moe_gmm_glu", "moe_gmm_glu_bwd_workspace_size",
           "moe_gmm_glu_bwd", "moe_gmm_dgrad", "moe_gmm_wgrad_workspace_size", "moe_gmm_wgrad", "moe_quant_mxfp4_rows", "moe_quant_mxfp4_weights",
           "moe_gmm_mxfp4_dyn_workspace_size", "moe_gmm_mxfp4_dyn", "moe_fetch_probe", "moe_mfma_probe")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built in-tree by build()); raise if it is not there."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libmoe.so not built at {LIB_PATH}; run __graft_entry__.build() "
                              "or python -m mixture_experts_layer_06_amd._build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_status_string.argtypes = [i32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_version.argtypes = []
        L.moe_version.restype = i32
        L.moe_route_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_route.argtypes = [vp, vp, i32, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]
        L.moe_permute_workspace_size.argtypes = [i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_permute.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_gmm_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_gmm.argtypes = [vp, i32, i32, vp, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32, vp,
                              i32, vp, sz, vp]
        L.moe_gmm_gather.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, i32, i32, vp, vp, i32, i32,
                                     i32, i32, i32, vp, i32, vp, sz, vp]
        L.moe_gmm_scatter.argtypes = [vp, i32, i32, vp, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32,
                                      vp, vp, vp, i32, vp, sz, vp]
        L.moe_gmm_routed_shared.argtypes = [vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp,
                                            vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
        L.moe_gmm_mx_routed_shared.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp,
                                               vp, i32, i32, i32, i32, i32, vp, vp]
        L.moe_gmm_mx.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
        L.moe_gmm_mxfp4.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
        L.moe_combine.argtypes = [vp, i32, vp, vp, i32, i32, i32, vp, i32, vp]
        L.moe_sum_slots.argtypes = [vp, i32, i32, i32, i32, vp, vp]
        L.moe_quant_rows.argtypes = [vp, i32, i32, i32, vp, i32, i32, vp, vp, vp]
        L.moe_layer_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_layer.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp,
                                vp, vp, sz, vp]
        L.moe_layer_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp,
                                        vp, vp]
        L.moe_layer_fp8_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_layer_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp,
                                    vp, sz, vp]
        L.moe_gmm_glu.argtypes = [vp, i32, vp, i32, i32, vp, vp, i32, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        L.moe_gmm_glu_bwd_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_gmm_glu_bwd.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, vp, vp, i32, vp, i32, i32, i32, i32, i32,
                                      vp, vp, vp, i32, vp, sz, vp]
        L.moe_gmm_dgrad.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, vp]
        L.moe_gmm_wgrad_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_gmm_wgrad.argtypes = [vp, i32, vp, i32, vp, i32, vp, i32, i32, i32, i32, vp, i32, vp, sz, vp]
        L.moe_quant_mxfp4_rows.argtypes = [vp, i32, i32, i32, vp, i32, i32, vp, vp, vp, vp]
        L.moe_quant_mxfp4_weights.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp]
        L.moe_gmm_mxfp4_dyn_workspace_size.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_gmm_mxfp4_dyn.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, sz, vp]
        L.moe_fetch_probe.argtypes = [vp, sz, i32, i32, i32, vp, vp]
        L.moe_mfma_probe.argtypes = [i32, i32, vp, vp, vp]
        for n in EXPORTS[2:]:
            getattr(L, n).restype = i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise MoeError(status, where)


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return FP8_E4M3
    raise TypeError(f"unsupported tensor dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr() if t.numel() else None


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


# ---------------------------------------------------------------- entry points

def route_workspace_size(T, H, E, K, dt) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_route_workspace_size(T, H, E, K, dt, ctypes.byref(n)), "moe_route_workspace_size")
    return n.value


def route(x, w_router, K, bias=None, topk_idx=None, topk_gate=None, ws=None, stream=None):
    """moe_route. Returns (topk_idx int32 (T,K), topk_gate fp32 (T,K)). ws: a device
    buffer of at least route_workspace_size() bytes, allocated here when None."""
    T, H = x.shape
    E = w_router.shape[1]
    dt = dtype_code(x)
    if topk_idx is None:
        topk_idx = _empty((T, K), torch.int32, x)
    if topk_gate is None:
        topk_gate = _empty((T, K), torch.float32, x)
    if ws is None:
        n = route_workspace_size(T, H, E, K, dt)
        ws = _empty((n,), torch.uint8, x) if n else None
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    st = lib().moe_route(_ptr(x), _ptr(w_router), dt, _ptr(bias), T, H, E, K,
                         _ptr(topk_idx), _ptr(topk_gate), _ptr(ws), nbytes, _stream(stream))
    _check(st, "moe_route")
    return topk_idx, topk_gate


def permute_workspace_size(T, E, K) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_permute_workspace_size(T, E, K, ctypes.byref(n)), "moe_permute_workspace_size")
    return n.value


def permute(topk_idx, E, x=None, ws=None, stream=None, out=None):
    """moe_permute. Returns dict counts, offsets, perm_src, perm_dst, x_perm (or None)."""
    T, K = topk_idx.shape
    A = T * K
    dev = topk_idx
    o = dict(out or {})
    counts = o.get("counts", _empty((E,), torch.int32, dev))
    offsets = o.get("offsets", _empty((E + 1,), torch.int32, dev))
    psrc = o.get("perm_src", _empty((A,), torch.int32, dev))
    pdst = o.get("perm_dst", _empty((A,), torch.int32, dev))
    xp = None
    H, dt = 1, F32
    if x is not None:
        H = x.shape[1]
        dt = dtype_code(x)
        xp = o.get("x_perm", _empty((A, H), x.dtype, dev))
    need = permute_workspace_size(T, E, K)
    if ws is None and need:
        ws = _empty((need,), torch.uint8, dev)
    st = lib().moe_permute(_ptr(topk_idx), _ptr(x), dt, T, H, E, K, _ptr(counts), _ptr(offsets),
                           _ptr(psrc), _ptr(pdst), _ptr(xp), _ptr(ws) if need else None,
                           ws.numel() if (ws is not None and need) else 0, _stream(stream))
    _check(st, "moe_permute")
    return {"counts": counts, "offsets": offsets, "perm_src": psrc, "perm_dst": pdst, "x_perm": xp}


def gmm_workspace_size(a_dt, e, A, Hin, N) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_gmm_workspace_size(a_dt, e, A, Hin, N, ctypes.byref(n)), "moe_gmm_workspace_size")
    return n.value


def gmm(a, w, offsets, act=ACT_NONE, a_scale=None, w_scale=None, out=None, ws=None, stream=None,
        rows=None, row_div=1, dst=None, gate=None, per_token=False):
    """moe_gmm over w (e,Hin,N). Scales (1-element fp32 device tensors) select
    MOE_QUANT_PER_TENSOR. Output: fp32 for fp32 inputs, else bf16. ws: a device
    buffer of at least gmm_workspace_size() bytes, allocated here when None.
    rows (int32 device tensor, one entry per grouped row): moe_gmm_gather, grouped
    row r is row rows[r] // row_div of a. dst (int32, one entry per grouped row):
    moe_gmm_scatter, grouped row r is stored as out row dst[r], times gate[dst[r]]
    when gate (fp32) is given. per_token: a_scale holds one fp32 per row of a
    (MOE_QUANT_PER_TOKEN, E4M3 activations)."""
    if dst is not None and rows is not None:
        raise ValueError("gather (rows) and scatter (dst) are separate entry points")
    A, Hin = a.shape
    if rows is not None:
        A = rows.numel()
    e, Hw, N = w.shape
    if Hw != Hin:
        raise ValueError("a and w disagree on Hin")
    adt, wdt = dtype_code(a), dtype_code(w)
    odt = F32 if adt == F32 else BF16
    if out is None:
        out = _empty((A, N), torch.float32 if odt == F32 else torch.bfloat16, a)
    if ws is None:
        n = gmm_workspace_size(adt, e, A, Hin, N)
        ws = _empty((n,), torch.uint8, a) if n else None
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    aq = QUANT_PER_TENSOR if a_scale is not None else QUANT_NONE
    if per_token:
        aq = QUANT_PER_TOKEN
    wq = QUANT_PER_TENSOR if w_scale is not None else QUANT_NONE
    if dst is not None:
        st = lib().moe_gmm_scatter(_ptr(a), adt, aq, _ptr(a_scale), _ptr(w), wdt, wq, _ptr(w_scale),
                                   _ptr(offsets), e, A, Hin, N, act, _ptr(dst), _ptr(gate), _ptr(out),
                                   odt, _ptr(ws), nbytes, _stream(stream))
        _check(st, "moe_gmm_scatter")
        return out
    if rows is not None:
        st = lib().moe_gmm_gather(_ptr(a), a.shape[0], _ptr(rows), row_div, adt, aq, _ptr(a_scale),
                                  _ptr(w), wdt, wq, _ptr(w_scale), _ptr(offsets), e, A, Hin, N, act,
                                  _ptr(out), odt, _ptr(ws), nbytes, _stream(stream))
        _check(st, "moe_gmm_gather")
        return out
    st = lib().moe_gmm(_ptr(a), adt, aq, _ptr(a_scale), _ptr(w), wdt, wq, _ptr(w_scale),
                       _ptr(offsets), e, A, Hin, N, act, _ptr(out), odt, _ptr(ws), nbytes,
                       _stream(stream))
    _check(st, "moe_gmm")
    return out


def gmm_routed_shared(a, w, offsets, a_scale, w_scale, xs, ws_w, offsets_s, act=ACT_NONE, act_s=ACT_NONE,
                      dst=None, gate=None, per_token=False, out=None, ys=None, stream=None):
    """moe_gmm_routed_shared: the E4M3 grouped GEMM over w (e,Hin,N) (per-tensor
    scales, or per_token: one a_scale per row of a; stored through dst, times
    gate, when dst is given) and the bf16 grouped GEMM xs @ ws_w (e_s,Hs,Ns)
    over offsets_s in one launch. Returns (out, ys), both bf16."""
    A, Hin = a.shape
    e, Hw, N = w.shape
    T, Hs = xs.shape
    e_s, Hw2, Ns = ws_w.shape
    if Hw != Hin or Hw2 != Hs:
        raise ValueError("activations and weights disagree on the reduction size")
    if out is None:
        out = _empty((A, N), torch.bfloat16, a)
    if ys is None:
        ys = _empty((T, Ns), torch.bfloat16, xs)
    aq = QUANT_PER_TOKEN if per_token else QUANT_PER_TENSOR
    st = lib().moe_gmm_routed_shared(_ptr(a), aq, _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(offsets), e, A,
                                     Hin, N, act, _ptr(dst), _ptr(gate), _ptr(out), _ptr(xs), _ptr(ws_w),
                                     _ptr(offsets_s), e_s, T, Hs, Ns, act_s, _ptr(ys), _stream(stream))
    _check(st, "moe_gmm_routed_shared")
    return out, ys


def gmm_mx_routed_shared(a, a_scale, w, w_scale, offsets, xs, ws_w, offsets_s, fp4=False, act=ACT_NONE,
                         act_s=ACT_NONE, out=None, ys=None, stream=None):
    """moe_gmm_mx_routed_shared: gmm_mx (fp4 False) or gmm_mxfp4 (fp4 True)
    and the bf16 grouped GEMM xs @ ws_w (e_s,Hs,Ns) over offsets_s in one
    launch. Returns (out, ys), both bf16."""
    A, Hb = a.shape
    Hin = 2 * Hb if fp4 else Hb
    e, Hw, N = w.shape
    T, Hs = xs.shape
    e_s, Hw2, Ns = ws_w.shape
    if Hw != Hb or Hw2 != Hs:
        raise ValueError("activations and weights disagree on the reduction size")
    if out is None:
        out = _empty((A, N), torch.bfloat16, a)
    if ys is None:
        ys = _empty((T, Ns), torch.bfloat16, xs)
    st = lib().moe_gmm_mx_routed_shared(_ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(offsets), e, A, Hin,
                                        N, act, int(bool(fp4)), _ptr(out), _ptr(xs), _ptr(ws_w), _ptr(offsets_s),
                                        e_s, T, Hs, Ns, act_s, _ptr(ys), _stream(stream))
    _check(st, "moe_gmm_mx_routed_shared")
    return out, ys


def gmm_mx(a, a_scale, w, w_scale, offsets, act=ACT_NONE, out=None, stream=None):
    """moe_gmm_mx: E4M3 a (A,Hin) and w (e,Hin,N) with E8M0 block scales a_scale
    (slice-major, (Hin/128, A, 4)) and w_scale (e,Hin/32,N) (uint8 device
    tensors); bf16 output."""
    A, Hin = a.shape
    e, Hw, N = w.shape
    if Hw != Hin:
        raise ValueError("a and w disagree on Hin")
    if out is None:
        out = _empty((A, N), torch.bfloat16, a)
    st = lib().moe_gmm_mx(_ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(offsets), e, A, Hin, N,
                          act, _ptr(out), _stream(stream))
    _check(st, "moe_gmm_mx")
    return out


def gmm_mxfp4(a, a_scale, w, w_scale, offsets, act=ACT_NONE, out=None, stream=None):
    """moe_gmm_mxfp4: E2M1 a (A, Hin/2) and w (e, Hin/2, N) packed bytes (two
    values per byte along Hin), E8M0 scales a_scale (slice-major, (Hin/256, A,
    8)) and w_scale (e, Hin/32, N) (uint8 device tensors); bf16 output."""
    A, Hh = a.shape
    e, Hw, N = w.shape
    if Hw != Hh:
        raise ValueError("a and w disagree on Hin")
    if out is None:
        out = _empty((A, N), torch.bfloat16, a)
    st = lib().moe_gmm_mxfp4(_ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(offsets), e, A, 2 * Hh, N,
                             act, _ptr(out), _stream(stream))
    _check(st, "moe_gmm_mxfp4")
    return out


def combine(y_perm, perm_dst, topk_gate, T, K, out=None, stream=None):
    """moe_combine: weighted sum (gate given) -> (T,N); Unpermute (gate None) -> (T*K,N)."""
    N = y_perm.shape[1]
    dt = dtype_code(y_perm)
    if out is None:
        shape = (T, N) if topk_gate is not None else (T * K, N)
        out = _empty(shape, y_perm.dtype, y_perm)
    st = lib().moe_combine(_ptr(y_perm), dt, _ptr(perm_dst), _ptr(topk_gate), T, K, N, _ptr(out),
                           dt, _stream(stream))
    _check(st, "moe_combine")
    return out


def quant_rows(x, rows=None, row_div=1, n_out=None, q=None, scale=None, stream=None):
    """moe_quant_rows: per-token dynamic E4M3 quantisation of x (f32/bf16,
    (x_rows,H)); output row r quantises x[rows[r] // row_div] (or x[r]).
    Returns (codes (R,H) float8_e4m3fn, scales (R,) fp32)."""
    x_rows, H = x.shape
    R = (rows.numel() if rows is not None else x_rows) if n_out is None else n_out
    if q is None:
        q = _empty((R, H), torch.float8_e4m3fn, x)
    if scale is None:
        scale = _empty((R,), torch.float32, x)
    st = lib().moe_quant_rows(_ptr(x), dtype_code(x), x_rows, H, _ptr(rows), row_div, R, _ptr(q), _ptr(scale),
                              _stream(stream))
    _check(st, "moe_quant_rows")
    return q, scale


def sum_slots(z, T, K, out=None, stream=None):
    """moe_sum_slots: y[t] = sum_k z[t*K+k] for z (T*K,N) -> (T,N)."""
    N = z.shape[1]
    dt = dtype_code(z)
    if out is None:
        out = _empty((T, N), z.dtype, z)
    _check(lib().moe_sum_slots(_ptr(z), dt, T, K, N, _ptr(out), _stream(stream)), "moe_sum_slots")
    return out


def layer_workspace_size(T, H, E, K, F, dtype_code_) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_layer_workspace_size(T, H, E, K, F, dtype_code_, ctypes.byref(n)),
           "moe_layer_workspace_size")
    return n.value


def layer(x, w_router, w1, w2, K, bias=None, act=ACT_RELU, y=None, ws=None, topk_idx=None,
          topk_gate=None, counts=None, stream=None):
    """moe_layer: route -> permute -> GEMM1(act) -> GEMM2 -> weighted combine. Returns y."""
    T, H = x.shape
    E, _, F = w1.shape
    dt = dtype_code(x)
    if y is None:
        y = torch.empty_like(x)
    need = layer_workspace_size(T, H, E, K, F, dt)
    if ws is None:
        ws = _empty((max(need, 1),), torch.uint8, x)
    st = lib().moe_layer(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w1), _ptr(w2), dt, T, H, E, K, F,
                         act, _ptr(y), _ptr(topk_idx), _ptr(topk_gate), _ptr(counts), _ptr(ws),
                         ws.numel(), _stream(stream))
    _check(st, "moe_layer")
    return y


def layer_noalloc(x, w_router, w1, w2, K, bias=None, act=ACT_RELU, y=None, topk_idx=None, topk_gate=None,
                  counts=None, stream=None):
    """moe_layer_noalloc: moe_layer with its scratch in the library's static
    device buffer (no workspace argument, nothing allocated by the call
    itself beyond y when y is None). Returns y."""
    T, H = x.shape
    E, _, F = w1.shape
    dt = dtype_code(x)
    if y is None:
        y = torch.empty_like(x)
    st = lib().moe_layer_noalloc(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w1), _ptr(w2), dt, T, H, E, K, F,
                                 act, _ptr(y), _ptr(topk_idx), _ptr(topk_gate), _ptr(counts), _stream(stream))
    _check(st, "moe_layer_noalloc")
    return y


def layer_fp8_workspace_size(T, H, E, K, F) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_layer_fp8_workspace_size(T, H, E, K, F, ctypes.byref(n)), "moe_layer_fp8_workspace_size")
    return n.value


def layer_fp8(x, w_router, w1, w1_scale, w2, w2_scale, K, bias=None, act=ACT_RELU, y=None, ws=None,
              topk_idx=None, topk_gate=None, counts=None, stream=None):
    """moe_layer_fp8: bf16 tokens x (T,H) and router (H,E); E4M3 experts w1
    (E,H,F), w2 (E,F,H) with one fp32 device scale each; bf16 y (T,H)."""
    T, H = x.shape
    E = w_router.shape[1]
    F = w1.shape[2]
    if y is None:
        y = _empty((T, H), torch.bfloat16, x)
    if ws is None:
        ws = _empty((layer_fp8_workspace_size(T, H, E, K, F),), torch.uint8, x)
    st = lib().moe_layer_fp8(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w1), _ptr(w1_scale), _ptr(w2),
                             _ptr(w2_scale), T, H, E, K, F, act, _ptr(y), _ptr(topk_idx), _ptr(topk_gate),
                             _ptr(counts), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_layer_fp8")
    return y


# ---------------------------------------------------------------- gated experts, gradients
#
# `stream` of the calls below: they run on it, and its inputs have to be ready
# there. Tensors that a call allocates may be used on the caller's current stream
# at once, which waits for them; with every output given it does not wait.

_STAY = contextlib.nullcontext()


def _launch_on(like, stream, *tensors):
    """Context of a call on `like`'s device: every tensor (None allowed) must
    live there. The device is made current and `stream` (default: the device's
    current one) too, so that buffers the call allocates belong to the stream
    that uses them; nothing changes where both are current already. Inputs have
    to be ready on `stream`; what the call allocates is ordered with the caller's
    stream by _hand_over."""
    dev = like.get_device()
    if dev < 0:
        raise ValueError("tensor must live on the GPU")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {t.device} and {like.device} in one call")
    if stream is None:
        return _STAY if dev == torch.cuda.current_device() else torch.cuda.device(dev)
    if stream.device != like.device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {like.device}")
    return torch.cuda.stream(stream)  # also makes the device current


def _hand_over(stream, *made):
    """Tensors a call allocated on `stream` (None among them allowed) become safe
    to use, and to drop, on the caller's current stream: it waits for them. With
    every output given nothing waits, and the streams stay apart."""
    made = [t for t in made if t is not None]
    if stream is None or not made:
        return
    here = torch.cuda.current_stream(stream.device)
    if here != stream:
        here.wait_stream(stream)
        for t in made:
            t.record_stream(here)


def _current(dev):
    """Handle of device dev's current stream. (current_stream() builds a Stream
    object on the way, 2.9 us where a small call takes 12.)"""
    return torch._C._cuda_getCurrentRawStream(dev)


def _dp(t):
    """Address of a dense tensor on the call's device; 0 (NULL) without elements."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _sizes(query, device, *args):
    """A workspace size query, asked once: it depends on its arguments and the
    (current) device only."""
    return query(*args)


def _check_like(name, t, dtype, shape, contiguous=True):
    if t is None:
        return
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_index(name, t, n):
    if t is not None and (t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries")


def _expert_matrix(name, w):
    """Data pointer and row stride of an expert weight tensor (e,Hin,N): dense, or
    a column range of a dense (e,Hin,ld) tensor."""
    if w.is_contiguous():
        return w.data_ptr(), w.shape[2]
    s0, s1, s2 = w.stride()
    if s2 != 1 or s0 != w.shape[1] * s1 or s1 < w.shape[2]:
        raise ValueError(f"{name} must be (e,Hin,N), contiguous or a column range of a contiguous tensor")
    return w.data_ptr(), s1


def _gate_up(w_gate, w_up, names=("w_gate", "w_up")):
    if w_gate.shape != w_up.shape or w_gate.dtype != w_up.dtype:
        raise ValueError(f"{names[0]} and {names[1]} must agree in shape and type")
    (pg, ld), (pu, ldu) = _expert_matrix(names[0], w_gate), _expert_matrix(names[1], w_up)
    if ld != ldu:
        raise ValueError(f"{names[0]} and {names[1]} must have the same strides")
    return pg, pu, ld


def _layer_dtype(t):
    dt = dtype_code(t)
    if dt == FP8_E4M3:
        raise TypeError(f"unsupported tensor dtype {t.dtype}")
    return dt


def _gmm_operands(x, w, offsets, rows):
    """(A, e, Hin, N) of rows x grouped by expert, checked against w and offsets."""
    e, Hin, N = w.shape
    if x.dim() != 2 or x.shape[1] != Hin or x.dtype != w.dtype:
        raise ValueError("x and the weights disagree on Hin or their type")
    A = x.shape[0] if rows is None else rows.numel()
    _check_index("rows", rows, A)
    _check_index("offsets", offsets, e + 1)
    return A, e, Hin, N


def gmm_glu(x, w_gate, w_up, offsets, act=ACT_SILU, rows=None, row_div=1, save=False, out=None, gate=None, up=None,
            stream=None):
    """moe_gmm_glu: act(x_r @ w_gate[e]) * (x_r @ w_up[e]) over rows grouped by
    expert; grouped row r is row r of x, or rows[r] // row_div of it. w_gate and
    w_up (e,Hin,N) are dense or the two halves of one dense (e,Hin,2N) tensor.
    Returns out (A,N); with save (or gate and up given) (out, gate, up), the
    projections moe_gmm_glu_bwd takes."""
    A, e, Hin, N = _gmm_operands(x, w_gate, offsets, rows)
    pg, pu, ld = _gate_up(w_gate, w_up)
    dt = _layer_dtype(x)
    dev = x.get_device()
    with _launch_on(x, stream, w_gate, w_up, offsets, rows, out, gate, up):
        if (gate is None) != (up is None):
            raise ValueError("gate and up come together")
        for name, t in (("out", out), ("gate", gate), ("up", up)):
            _check_like(name, t, x.dtype, (A, N))
        save = save or gate is not None
        made = []
        if out is None:
            out = _empty((A, N), x.dtype, x)
            made.append(out)
        if save and gate is None:
            gate, up = _empty((A, N), x.dtype, x), _empty((A, N), x.dtype, x)
            made += (gate, up)
        st = lib().moe_gmm_glu(_dp(x), x.shape[0], _dp(rows), row_div, dt, pg, pu, ld, _dp(offsets), e, A, Hin, N,
                               act, _dp(out), _dp(gate) if save else None, _dp(up) if save else None, _current(dev))
    _check(st, "moe_gmm_glu")
    _hand_over(stream, *made)
    return (out, gate, up) if save else out


def gmm_glu_bwd_workspace_size(dt, e, A, Hin, N) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_gmm_glu_bwd_workspace_size(dt, e, A, Hin, N, ctypes.byref(n)), "moe_gmm_glu_bwd_workspace_size")
    return n.value


def gmm_glu_bwd(dout, gate, up, x, w_gate, w_up, offsets, act=ACT_SILU, rows=None, row_div=1, need_da=True,
                need_dw=True, da=None, dw_gate=None, dw_up=None, ws=None, stream=None):
    """moe_gmm_glu_bwd: the gradients of gmm_glu for its grouped rows, da (A,Hin),
    and its weights, dw_gate and dw_up (e,Hin,N) (given, they may be column
    ranges of one dense tensor; allocated here they are so where w_gate and w_up
    are). need_da / need_dw False leave a gradient out (None is returned for it).
    A token's gradient is the sum over its rows: combine(da, perm_dst, ones, T, K)."""
    A, e, Hin, N = _gmm_operands(x, w_gate, offsets, rows)
    pg, pu, ld = _gate_up(w_gate, w_up)
    dt = _layer_dtype(x)
    dev = x.get_device()
    with _launch_on(x, stream, dout, gate, up, w_gate, w_up, offsets, rows, da, dw_gate, dw_up, ws):
        for name, t in (("dout", dout), ("gate", gate), ("up", up)):
            _check_like(name, t, x.dtype, (A, N))
        if (dw_gate is None) != (dw_up is None):
            raise ValueError("dw_gate and dw_up come together")
        _check_like("da", da, x.dtype, (A, Hin))
        _check_like("dw_gate", dw_gate, x.dtype, (e, Hin, N), contiguous=False)
        made = []
        if not need_da:
            da = None
        elif da is None:
            da = _empty((A, Hin), x.dtype, x)
            made.append(da)
        pdg = pdu = None
        lddw = N
        if not need_dw:
            dw_gate = dw_up = None
        elif dw_gate is not None:
            pdg, pdu, lddw = _gate_up(dw_gate, dw_up, ("dw_gate", "dw_up"))
        elif ld == 2 * N and pu - pg == N * w_gate.element_size():
            dw = _empty((e, Hin, 2 * N), x.dtype, x)
            made.append(dw)
            dw_gate, dw_up = dw[:, :, :N], dw[:, :, N:]
            pdg, pdu, lddw = dw_gate.data_ptr(), dw_up.data_ptr(), 2 * N
        else:
            dw_gate, dw_up = _empty((e, Hin, N), x.dtype, x), _empty((e, Hin, N), x.dtype, x)
            made += (dw_gate, dw_up)
            pdg, pdu = dw_gate.data_ptr(), dw_up.data_ptr()
        if ws is None:
            ws = _empty((_sizes(gmm_glu_bwd_workspace_size, dev, dt, e, A, Hin, N),), torch.uint8, x)
        st = lib().moe_gmm_glu_bwd(_dp(dout), _dp(gate), _dp(up), _dp(x), x.shape[0], _dp(rows), row_div, dt, pg,
                                   pu, ld, _dp(offsets), e, A, Hin, N, act, _dp(da), pdg, pdu, lddw, _dp(ws),
                                   ws.numel() * ws.element_size(), _current(dev))
    _check(st, "moe_gmm_glu_bwd")
    _hand_over(stream, *made)
    return da, dw_gate, dw_up


def gmm_dgrad(dout, w, offsets, out=None, stream=None):
    """moe_gmm_dgrad: da[r] = dout[r] @ w[e].T over rows grouped by expert; dout (A,N),
    w (e,Hin,N). Returns da (A,Hin)."""
    e, Hin, N = w.shape
    A = dout.shape[0]
    dt = _layer_dtype(w)
    _check_like("dout", dout, w.dtype, (A, N))
    _check_index("offsets", offsets, e + 1)
    dev = w.get_device()
    with _launch_on(w, stream, dout, offsets, out):
        made = out is None
        if made:
            out = _empty((A, Hin), w.dtype, w)
        _check_like("out", out, w.dtype, (A, Hin))
        st = lib().moe_gmm_dgrad(_dp(dout), dt, _dp(w), _dp(offsets), e, A, Hin, N, _dp(out), _current(dev))
    _check(st, "moe_gmm_dgrad")
    _hand_over(stream, out if made else None)
    return out


def gmm_wgrad_workspace_size(dt, e, A, Hin, N) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_gmm_wgrad_workspace_size(dt, e, A, Hin, N, ctypes.byref(n)), "moe_gmm_wgrad_workspace_size")
    return n.value


def gmm_wgrad(x, dout, offsets, rows=None, row_div=1, out=None, out_dtype=None, ws=None, stream=None):
    """moe_gmm_wgrad: dw[e] = x_r.T @ dout over each expert's rows; grouped row r is
    row r of x, or rows[r] // row_div of it; dout (A,N). Returns dw (e,Hin,N) in
    x's type, or float32 (out_dtype)."""
    A, N = dout.shape
    Hin = x.shape[1]
    e = offsets.numel() - 1
    dt = _layer_dtype(x)
    _check_like("dout", dout, x.dtype, (x.shape[0] if rows is None else rows.numel(), N))
    _check_index("rows", rows, A)
    _check_index("offsets", offsets, e + 1)
    dev = x.get_device()
    with _launch_on(x, stream, dout, offsets, rows, out, ws):
        made = out is None
        if made:
            out = _empty((e, Hin, N), out_dtype or x.dtype, x)
        _check_like("out", out, out_dtype or out.dtype, (e, Hin, N))
        if ws is None:
            n = _sizes(gmm_wgrad_workspace_size, dev, dt, e, A, Hin, N)
            ws = _empty((n,), torch.uint8, x) if n else None
        nbytes = ws.numel() * ws.element_size() if ws is not None else 0
        st = lib().moe_gmm_wgrad(_dp(x), x.shape[0], _dp(rows), row_div, _dp(dout), dt, _dp(offsets), e, A, Hin, N,
                                 _dp(out), _layer_dtype(out), _dp(ws), nbytes, _current(dev))
    _check(st, "moe_gmm_wgrad")
    _hand_over(stream, out if made else None)
    return out


def quant_mxfp4_rows(x, rows=None, row_div=1, n_out=None, codes=True, q=None, scale=None, values=False, stream=None):
    """moe_quant_mxfp4_rows: MXFP4 codes and scales of the rows of x (x_rows,H);
    output row r is row rows[r] // row_div of x (or row r). Returns (q (R,H/2)
    uint8, scale (H/256,R,8) uint8), and with values (True, or a bf16 tensor to
    fill) the numbers they stand for, bf16 (R,H). codes False: values only,
    (None, None, values)."""
    x_rows, H = x.shape
    R = (rows.numel() if rows is not None else x_rows) if n_out is None else n_out
    dt = _layer_dtype(x)
    given = values if isinstance(values, torch.Tensor) else None
    dev = x.get_device()
    with _launch_on(x, stream, rows, q, scale, given):
        _check_index("rows", rows, R)
        made = []
        if codes and q is None:
            q = _empty((R, H // 2), torch.uint8, x)
            made.append(q)
        if codes and scale is None:
            scale = _empty((H // 256, R, 8), torch.uint8, x)
            made.append(scale)
        v = given
        if v is None and values:
            v = _empty((R, H), torch.bfloat16, x)
            made.append(v)
        if not codes:
            q = scale = None
        _check_like("q", q, torch.uint8, (R, H // 2))
        _check_like("scale", scale, torch.uint8, (H // 256, R, 8))
        _check_like("values", v, torch.bfloat16, (R, H))
        st = lib().moe_quant_mxfp4_rows(_dp(x), dt, x_rows, H, _dp(rows), row_div, R, _dp(q), _dp(scale), _dp(v),
                                        _current(dev))
    _check(st, "moe_quant_mxfp4_rows")
    _hand_over(stream, *made)
    return (q, scale, v) if v is not None else (q, scale)


def quant_mxfp4_weights(w, codes=True, q=None, scale=None, values=False, stream=None):
    """moe_quant_mxfp4_weights: MXFP4 codes and scales of expert weights w (e,Hin,N),
    blocks along Hin, as moe_gmm_mxfp4 takes them. Returns (q (e,Hin/2,N) uint8,
    scale (e,Hin/32,N64) uint8), and with values (True, or a bf16 tensor to fill)
    the numbers they stand for, bf16 (e,Hin,N). codes False: (None, None, values)."""
    e, Hin, N = w.shape
    n64 = (N + 63) // 64 * 64
    dt = _layer_dtype(w)
    given = values if isinstance(values, torch.Tensor) else None
    dev = w.get_device()
    with _launch_on(w, stream, q, scale, given):
        made = []
        if codes and q is None:
            q = _empty((e, Hin // 2, N), torch.uint8, w)
            made.append(q)
        if codes and scale is None:
            scale = _empty((e, Hin // 32, n64), torch.uint8, w)
            made.append(scale)
        v = given
        if v is None and values:
            v = _empty((e, Hin, N), torch.bfloat16, w)
            made.append(v)
        if not codes:
            q = scale = None
        _check_like("q", q, torch.uint8, (e, Hin // 2, N))
        _check_like("scale", scale, torch.uint8, (e, Hin // 32, n64))
        _check_like("values", v, torch.bfloat16, (e, Hin, N))
        st = lib().moe_quant_mxfp4_weights(_dp(w), dt, e, Hin, N, _dp(q), _dp(scale), _dp(v), _current(dev))
    _check(st, "moe_quant_mxfp4_weights")
    _hand_over(stream, *made)
    return (q, scale, v) if v is not None else (q, scale)


def gmm_mxfp4_dyn_workspace_size(e, A, Hin, N) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_gmm_mxfp4_dyn_workspace_size(e, A, Hin, N, ctypes.byref(n)), "moe_gmm_mxfp4_dyn_workspace_size")
    return n.value


def gmm_mxfp4_dyn(x, w, w_scale, offsets, act=ACT_NONE, rows=None, row_div=1, out=None, ws=None, stream=None):
    """moe_gmm_mxfp4_dyn: rows of x (f32 or bf16, (x_rows,Hin)) quantised to MXFP4 in
    the call, times MXFP4 expert weights w (e,Hin/2,N) with w_scale; grouped row r
    is row rows[r] // row_div of x (or row r). Returns bf16 (A,N)."""
    x_rows, Hin = x.shape
    e, Hh, N = w.shape
    A = x_rows if rows is None else rows.numel()
    dt = _layer_dtype(x)
    if Hin != 2 * Hh:
        raise ValueError("x and w disagree on Hin")
    dev = x.get_device()
    with _launch_on(x, stream, w, w_scale, offsets, rows, out, ws):
        _check_like("w", w, torch.uint8, (e, Hh, N))
        _check_like("w_scale", w_scale, torch.uint8, (e, Hin // 32, (N + 63) // 64 * 64))
        _check_index("rows", rows, A)
        _check_index("offsets", offsets, e + 1)
        made = out is None
        if made:
            out = _empty((A, N), torch.bfloat16, x)
        _check_like("out", out, torch.bfloat16, (A, N))
        if ws is None:
            n = _sizes(gmm_mxfp4_dyn_workspace_size, dev, e, A, Hin, N)
            ws = _empty((n,), torch.uint8, x) if n else None
        nbytes = ws.numel() * ws.element_size() if ws is not None else 0
        st = lib().moe_gmm_mxfp4_dyn(_dp(x), dt, x_rows, _dp(rows), row_div, _dp(w), _dp(w_scale), _dp(offsets), e,
                                     A, Hin, N, act, _dp(out), _dp(ws), nbytes, _current(dev))
    _check(st, "moe_gmm_mxfp4_dyn")
    _hand_over(stream, out if made else None)
    return out


def fetch_probe(buf, mode, shared_window, kb_per_wave, stream=None, cycles=None):
    """moe_fetch_probe over the uint8 device tensor buf (mode 0: LDS DMA, 1:
    vector loads). Returns the per-compute-unit s_memtime ticks (int64
    device tensor, one entry per CU; pass `cycles` to reuse one, so that a
    timed call launches nothing else) and the bytes each CU read; time the
    call with stream events for a rate."""
    ncu = torch.cuda.get_device_properties(buf.device).multi_processor_count
    if cycles is None:
        cycles = torch.zeros((ncu,), dtype=torch.int64, device=buf.device)
    elif cycles.numel() != ncu or cycles.dtype != torch.int64 or cycles.device != buf.device:
        raise ValueError("cycles must be an int64 tensor of one entry per compute unit on buf's device")
    _check(lib().moe_fetch_probe(_ptr(buf), buf.numel(), mode, 1 if shared_window else 0, kb_per_wave,
                                 _ptr(cycles), _stream(stream)), "moe_fetch_probe")
    return cycles, 8 * kb_per_wave * 1024


def mfma_probe(fp8, iters, device="cuda", stream=None, cycles=None, sink=None):
    """moe_mfma_probe: per-CU s_memtime ticks (int64 device tensor) and the
    flops each CU issued; pass `cycles` (int64, one per CU) and `sink`
    (float32, 512 per CU) to reuse them, so that a timed call launches
    nothing else; time the call with stream events for a rate."""
    ncu = torch.cuda.get_device_properties(torch.device(device)).multi_processor_count
    if cycles is None:
        cycles = torch.zeros((ncu,), dtype=torch.int64, device=device)
    if sink is None:
        sink = torch.empty((ncu * 512,), dtype=torch.float32, device=device)
    if cycles.numel() != ncu or cycles.dtype != torch.int64 or sink.numel() < ncu * 512 or sink.dtype != torch.float32:
        raise ValueError("cycles: int64, one per compute unit; sink: float32, 512 per compute unit")
    _check(lib().moe_mfma_probe(FP8_E4M3 if fp8 else BF16, iters, _ptr(sink), _ptr(cycles), _stream(stream)),
           "moe_mfma_probe")
    return cycles, 8 * 8 * iters * (131072 if fp8 else 16384)
