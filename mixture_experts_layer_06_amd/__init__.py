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
NORM_RMS, NORM_LAYER = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2

EXPORTS = ("moe_status_string", "moe_version", "moe_route_workspace_size", "moe_route",
           "moe_permute_workspace_size", "moe_permute", "moe_gmm_workspace_size", "moe_gmm",
           "moe_gmm_gather", "moe_gmm_scatter", "moe_gmm_routed_shared", "moe_gmm_mx_routed_shared", "moe_gmm_mx", "moe_gmm_mxfp4", "moe_combine", "moe_sum_slots",
           "moe_quant_rows", "moe_layer_workspace_size", "moe_layer", "moe_layer_fp8_workspace_size",
           "moe_layer_fp8", "moe_layer_noalloc", "moe_gmm_glu", "moe_gmm_glu_bwd_workspace_size",
           "moe_gmm_glu_bwd", "moe_gmm_dgrad", "moe_gmm_wgrad_workspace_size", "moe_gmm_wgrad", "moe_quant_mxfp4_rows", "moe_quant_mxfp4_weights",
           "moe_gmm_mxfp4_dyn_workspace_size", "moe_gmm_mxfp4_dyn", "moe_route_scores",
           "moe_router_loss_workspace_size", "moe_router_loss", "moe_router_loss_bwd", "moe_combine_bwd",
           "moe_block_norm", "moe_block_norm_bwd_workspace_size", "moe_block_norm_bwd", "moe_lora_workspace_size",
           "moe_lora", "moe_lora_filled", "moe_lora_bwd_workspace_size", "moe_lora_bwd", "moe_lora_bwd_filled",
           "moe_fetch_probe", "moe_mfma_probe")


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
        psz, f32 = ctypes.POINTER(sz), ctypes.c_float
        L.moe_route_scores.argtypes = [vp, vp, i32, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
        L.moe_router_loss_workspace_size.argtypes = [i32, i32, i32, psz]
        L.moe_router_loss.argtypes = [vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_router_loss_bwd.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp]
        L.moe_combine_bwd.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp]
        L.moe_block_norm.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp, i32, f32, f32, f32,
                                     vp, vp, vp]
        L.moe_block_norm_bwd_workspace_size.argtypes = [i32, i32, psz]
        L.moe_block_norm_bwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, i32, vp, i32, f32,
                                         f32, f32, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
        L.moe_lora_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, psz]
        L.moe_lora.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, sz, vp]
        L.moe_lora_filled.argtypes = L.moe_lora.argtypes
        L.moe_lora_bwd_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, psz]
        L.moe_lora_bwd.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp,
                                   i32, vp, sz, vp]
        L.moe_lora_bwd_filled.argtypes = L.moe_lora_bwd.argtypes
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


def route(x, w_router, K, bias=None, topk_idx=None, topk_gate=None, ws=None, stream=None, scores=None):
    """moe_route. Returns (topk_idx int32 (T,K), topk_gate fp32 (T,K)). ws: a device
    buffer of at least route_workspace_size() bytes, allocated here when None. scores
    (True, or an fp32 (T,E) tensor to fill): moe_route_scores, a third result, the
    scores that were ranked."""
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
    if scores is not None and scores is not False:
        if scores is True:
            scores = _empty((T, E), torch.float32, x)
        _check_like("scores", scores, torch.float32, (T, E))
        st = lib().moe_route_scores(_ptr(x), _ptr(w_router), dt, _ptr(bias), T, H, E, K, _ptr(topk_idx),
                                    _ptr(topk_gate), _ptr(scores), _ptr(ws), nbytes, _stream(stream))
        _check(st, "moe_route_scores")
        return topk_idx, topk_gate, scores
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


def _nbytes(t):
    return t.numel() * t.element_size() if t is not None else 0


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


# ---------------------------------------------------------------- router losses, the combine's gradient

def router_loss_workspace_size(T, E, K) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_router_loss_workspace_size(T, E, K, ctypes.byref(n)), "moe_router_loss_workspace_size")
    return n.value


def _check_mask(mask, T):
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.shape != (T,)
                             or not mask.is_contiguous()):
        raise ValueError(f"mask must be a contiguous bool or uint8 tensor of {T} entries")


def router_loss(scores, topk_idx, mask=None, counts=None, tokens=None, probs=None, loss=None, ws=None, stream=None):
    """moe_router_loss: per-expert counts and the balance and z losses of scores (T,E)
    and the chosen experts topk_idx (T,K); mask (T): False for tokens that do not
    count. Returns dict loss fp32 (2) [balance, z], counts int32 (E), tokens int32
    (1), probs fp32 (E)."""
    T, E = scores.shape
    K = topk_idx.shape[1]
    dt = _layer_dtype(scores)
    dev = scores.get_device()
    with _launch_on(scores, stream, topk_idx, mask, counts, tokens, probs, loss, ws):
        _check_like("scores", scores, scores.dtype, (T, E))
        _check_like("topk_idx", topk_idx, torch.int32, (T, K))
        _check_mask(mask, T)
        made = []
        if counts is None:
            counts = scores.new_empty(E, dtype=torch.int32)
            made.append(counts)
        if tokens is None:
            tokens = scores.new_empty(1, dtype=torch.int32)
            made.append(tokens)
        if probs is None:
            probs = scores.new_empty(E, dtype=torch.float32)
            made.append(probs)
        if loss is None:
            loss = scores.new_empty(2, dtype=torch.float32)
            made.append(loss)
        if len(made) < 4:
            _check_like("counts", counts, torch.int32, (E,))
            _check_like("tokens", tokens, torch.int32, (1,))
            _check_like("probs", probs, torch.float32, (E,))
            _check_like("loss", loss, torch.float32, (2,))
        if ws is None:
            n = _sizes(router_loss_workspace_size, dev, T, E, K)
            ws = _empty((n,), torch.uint8, scores) if n else None
        st = lib().moe_router_loss(_dp(scores), dt, _dp(topk_idx), _dp(mask), T, E, K, _dp(counts), _dp(tokens),
                                   _dp(probs), _dp(loss), _dp(ws), _nbytes(ws), _current(dev))
    _check(st, "moe_router_loss")
    _hand_over(stream, *made)
    return {"loss": loss, "counts": counts, "tokens": tokens, "probs": probs}


def router_loss_bwd(scores, topk_idx, counts=None, tokens=None, dloss=None, gate=None, dgate=None, mask=None,
                    out=None, out_dtype=None, stream=None):
    """moe_router_loss_bwd: the gradient of scores (T,E), from dloss fp32 (2), the
    gradients of router_loss's losses (with its counts and tokens), and from dgate
    fp32 (T,K), that of the kept gates `gate`; either may be left out. Returns (T,E)
    in out_dtype (default: that of scores)."""
    T, E = scores.shape
    K = topk_idx.shape[1]
    dt = _layer_dtype(scores)
    dev = scores.get_device()
    with _launch_on(scores, stream, topk_idx, counts, tokens, dloss, gate, dgate, mask, out):
        _check_like("scores", scores, scores.dtype, (T, E))
        _check_like("topk_idx", topk_idx, torch.int32, (T, K))
        _check_like("counts", counts, torch.int32, (E,))
        _check_like("tokens", tokens, torch.int32, (1,))
        _check_like("dloss", dloss, torch.float32, (2,))
        _check_like("gate", gate, torch.float32, (T, K))
        _check_like("dgate", dgate, torch.float32, (T, K))
        _check_mask(mask, T)
        made = out is None
        if made:
            out = torch.empty_like(scores, dtype=out_dtype)
        else:
            _check_like("out", out, out_dtype or out.dtype, (T, E))
        st = lib().moe_router_loss_bwd(_dp(scores), dt, _dp(topk_idx), _dp(mask), _dp(counts), _dp(tokens),
                                       _dp(dloss), _dp(gate), _dp(dgate), T, E, K, _dp(out), _layer_dtype(out),
                                       _current(dev))
    _check(st, "moe_router_loss_bwd")
    _hand_over(stream, out if made else None)
    return out


def combine_bwd(dout, y_perm, perm_dst, topk_gate, need_dy=True, need_dgate=True, dy_perm=None, dgate=None,
                stream=None):
    """moe_combine_bwd: the gradient of combine (with gates) for its rows, dy_perm
    (T*K,N), and its gates, dgate fp32 (T,K); need_* False leaves one out (None). A row
    that no entry of perm_dst names (entries outside [0, T*K), of dropped slots) is not
    written: where there are such, give a dy_perm that holds what they should."""
    T, N = dout.shape
    K = topk_gate.shape[1]
    dt = _layer_dtype(dout)
    dev = dout.get_device()
    with _launch_on(dout, stream, y_perm, perm_dst, topk_gate, dy_perm, dgate):
        _check_like("dout", dout, dout.dtype, (T, N))
        _check_like("y_perm", y_perm, dout.dtype, (T * K, N))
        _check_index("perm_dst", perm_dst, T * K)
        _check_like("topk_gate", topk_gate, torch.float32, (T, K))
        made = []
        if not need_dy:
            dy_perm = None
        elif dy_perm is None:
            dy_perm = dout.new_empty((T * K, N)) if y_perm is None else torch.empty_like(y_perm)
            made.append(dy_perm)
        if not need_dgate:
            dgate = None
        elif dgate is None:
            dgate = torch.empty_like(topk_gate)
            made.append(dgate)
        _check_like("dy_perm", dy_perm, dout.dtype, (T * K, N))
        _check_like("dgate", dgate, torch.float32, (T, K))
        st = lib().moe_combine_bwd(_dp(dout), _dp(y_perm), dt, _dp(perm_dst), _dp(topk_gate), T, K, N, _dp(dy_perm),
                                   _dp(dgate), _current(dev)) if T else OK
    _check(st, "moe_combine_bwd")
    _hand_over(stream, *made)
    return dy_perm, dgate


# ---------------------------------------------------------------- norms around a block

def _gate_mode(gate, T, N):
    if gate is None:
        return GATE_NONE
    if gate.shape == (N,):
        return GATE_CHANNEL
    if gate.shape == (T, 1):
        return GATE_TOKEN
    raise ValueError(f"gate must be ({N},) per channel or ({T}, 1) per token, got {tuple(gate.shape)}")


def _norm_weights(N, named, gate):
    """Type of the weights, biases and gate, which share one (float32 without any)."""
    given = [t for _, t in named if t is not None] + ([gate] if gate is not None else [])
    wt = given[0].dtype if given else torch.float32
    for name, t in named:
        _check_like(name, t, wt, (N,))
    if gate is not None:
        _check_like("gate", gate, wt, gate.shape)
    return wt


_CODE = {torch.float32: F32, torch.bfloat16: BF16}


def block_norm(z, r, w_post=None, b_post=None, gate=None, w_pre=None, b_pre=None, post=None, pre=True, alpha=1.0,
               beta=1.0, eps=1e-6, kind=NORM_RMS, r_out=None, h=None, stream=None):
    """moe_block_norm: r_out = alpha * r + beta * gate * post(z), h = pre(r_out).
    z (T,N): the block's output; r (T,N) or None: the residual stream, of z's type or
    float32. post: whether z is normalised (default: w_post is given); pre False: no
    h. gate: (N,) per channel or (T,1) per token. z None: h is the norm of r alone.
    Returns (r_out, h), None for what there is not."""
    like = r if z is None else z
    if like is None:
        raise ValueError("block_norm needs z or r")
    T, N = like.shape
    dt_t = like.dtype if h is None or z is not None else h.dtype
    r_t = r.dtype if r is not None else r_out.dtype if r_out is not None else dt_t
    post = w_post is not None if post is None else bool(post)
    dt = _layer_dtype(like)
    dev = like.get_device()
    with _launch_on(like, stream, z, r, w_post, b_post, gate, w_pre, b_pre, r_out, h):
        _check_like("z", z, dt_t, (T, N))
        _check_like("r", r, r_t, (T, N))
        wt = _norm_weights(N, (("w_post", w_post), ("b_post", b_post), ("w_pre", w_pre), ("b_pre", b_pre)), gate)
        made = []
        if z is not None and r_out is None:
            r_out = torch.empty_like(like if r is None else r)
            made.append(r_out)
        else:
            _check_like("r_out", r_out, r_t, (T, N))
        if not pre:
            h = None
        elif h is None:
            h = torch.empty_like(like)
            made.append(h)
        else:
            _check_like("h", h, dt_t, (T, N))
        st = lib().moe_block_norm(_dp(z), _dp(r), _CODE.get(dt_t, -1), _CODE.get(r_t, -1), T, N, kind, int(post),
                                  _dp(w_post), _dp(b_post), _dp(gate), _gate_mode(gate, T, N), _dp(w_pre),
                                  _dp(b_pre), _CODE.get(wt, -1), alpha, beta, eps, _dp(r_out), _dp(h), _current(dev))
    _check(st, "moe_block_norm")
    _hand_over(stream, *made)
    return r_out, h


def block_norm_bwd_workspace_size(T, N) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_block_norm_bwd_workspace_size(T, N, ctypes.byref(n)), "moe_block_norm_bwd_workspace_size")
    return n.value


def block_norm_bwd(dh, dr_out, z, r_out, w_post=None, b_post=None, gate=None, w_pre=None, post=None, alpha=1.0,
                   beta=1.0, eps=1e-6, kind=NORM_RMS, need_dr=True, need_dz=True, need_dw=True, dw_dtype=None, dr=None,
                   dz=None, ws=None, stream=None, b_pre=None):
    """moe_block_norm_bwd: the gradients of block_norm. dh: that of h, None without h;
    dr_out: that of r_out from its other readers, or None; z, r_out as they were.
    Returns a dict of dr, dz (without z: dr alone), dw_post, dw_pre and dgate for those
    given, and for layer norms db_post and db_pre where the norm's weight or its bias
    is (b_pre has no other part in the gradients); weights' gradients in dw_dtype
    (default: theirs). need_* False leaves gradients out (need_dw: those of weights,
    biases and gate)."""
    like = z if z is not None else r_out if r_out is not None else dr_out
    if like is None:
        raise ValueError("block_norm_bwd needs z or r_out")
    T, N = like.shape
    dt_t = z.dtype if z is not None else dh.dtype if dh is not None else like.dtype
    r_t = r_out.dtype if r_out is not None else dr_out.dtype if dr_out is not None else dt_t
    post = w_post is not None if post is None else bool(post)
    _layer_dtype(like)
    dev = like.get_device()
    if b_pre is not None and (kind != NORM_LAYER or dh is None):
        raise MoeError(ERR_UNSUPPORTED, "moe_block_norm_bwd")  # RMS norms have no bias; nor is there one without dh
    with _launch_on(like, stream, dh, dr_out, z, r_out, w_post, b_post, gate, w_pre, b_pre, dr, dz, ws):
        for name, t, dtype in (("dh", dh, dt_t), ("dr_out", dr_out, r_t), ("z", z, dt_t), ("r_out", r_out, r_t)):
            _check_like(name, t, dtype, (T, N))
        wt = _norm_weights(N, (("w_post", w_post), ("b_post", b_post), ("w_pre", w_pre), ("b_pre", b_pre)), gate)
        dwt = dw_dtype or wt
        mode = _gate_mode(gate, T, N)
        made, out = [], {}

        def new(name, shape, dtype):
            out[name] = like.new_empty(shape, dtype=dtype)
            made.append(out[name])

        for name, need, given, dtype in (("dr", need_dr, dr, r_t), ("dz", need_dz and z is not None, dz, dt_t)):
            if need and given is None:
                new(name, (T, N), dtype)
            elif need:
                _check_like(name, given, dtype, (T, N))
                out[name] = given
        if need_dw:
            for side, w, b, there in (("post", w_post, b_post, post), ("pre", w_pre, b_pre, dh is not None)):
                if w is not None and there:
                    new("dw_" + side, (N,), dwt)
                if kind == NORM_LAYER and there and (w is not None or b is not None):
                    new("db_" + side, (N,), dwt)
            if gate is not None:
                new("dgate", gate.shape, dwt)
        sums = any(k[:2] in ("dw", "db") for k in out) or mode == GATE_CHANNEL and "dgate" in out
        if ws is None and sums:
            ws = _empty((_sizes(block_norm_bwd_workspace_size, dev, T, N),), torch.uint8, like)
        st = lib().moe_block_norm_bwd(_dp(dh), _dp(dr_out), _dp(z), _dp(r_out), _CODE.get(dt_t, -1),
                                      _CODE.get(r_t, -1), T, N, kind, int(post), _dp(w_post), _dp(b_post), _dp(gate),
                                      mode, _dp(w_pre), _CODE.get(wt, -1), alpha, beta, eps,
                                      *(_dp(out.get(k)) for k in ("dr", "dz", "dw_post", "db_post", "dgate",
                                                                  "dw_pre", "db_pre")),
                                      _CODE.get(dwt, -1), _dp(ws), _nbytes(ws), _current(dev))
    _check(st, "moe_block_norm_bwd")
    _hand_over(stream, *made)
    return out


# ---------------------------------------------------------------- low-rank adapters

def lora_workspace_size(dt, e, M, H, N, R) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_lora_workspace_size(dt, e, M, H, N, R, ctypes.byref(n)), "moe_lora_workspace_size")
    return n.value


def lora_bwd_workspace_size(dt, e, M, H, N, R) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_lora_bwd_workspace_size(dt, e, M, H, N, R, ctypes.byref(n)), "moe_lora_bwd_workspace_size")
    return n.value


def _lora_shapes(T, width, side, a, b, offsets, rows, scale):
    e, H, R = a.shape
    N = b.shape[2]
    _check_like("a", a, a.dtype, (e, H, R))
    _check_like("b", b, a.dtype, (e, R, N))
    if width != (H if side == "x" else N):
        raise ValueError(f"{side} and the adapters disagree on its width")
    M = T if rows is None else rows.numel()
    _check_index("rows", rows, M)
    _check_index("offsets", offsets, e + 1)
    _check_like("scale", scale, torch.float32, (e,))
    return e, M, H, N, R


def _beside(base, out, shape, like, M, rows, made):
    """Base and output of an adapter call, and whether the call has to fill the rows that
    `rows` does not list. Without `out` that is a new tensor, which starts as base (or
    zeros) where the list is shorter than it; a list as long may still name fewer rows."""
    fill = False
    if out is None:
        if M < shape[0]:
            out = base.clone() if base is not None else torch.zeros(shape, dtype=like.dtype, device=like.device)
            base = out if base is not None else None
        else:
            out = _empty(shape, like.dtype, like)
            fill = rows is not None
        made.append(out)
    _check_like("base", base, like.dtype, shape)
    return base, out, fill


def lora(x, a, b, offsets, rows=None, scale=None, base=None, out=None, u=None, ws=None, stream=None):
    """moe_lora: base[t] + scale[e] * (x[t] @ a[e]) @ b[e] over rows grouped by adapter;
    grouped row r is row t = rows[r] of x (T,H) and base (T,N), or row r. a (e,H,R),
    b (e,R,N). out may be base itself (rows of no adapter, and rows that are not
    listed, stay as they are there; a new tensor has base, or zeros, in them). u: True, or an fp32 (M,R) tensor to fill: also returns
    x @ a of the grouped rows, what lora_bwd takes."""
    T, H = x.shape
    dev = x.get_device()
    dt = _layer_dtype(x)
    with _launch_on(x, stream, a, b, offsets, rows, scale, base, out, ws, u if u is not True else None):
        e, M, H, N, R = _lora_shapes(T, H, "x", a, b, offsets, rows, scale)
        _check_like("x", x, a.dtype, (T, H))
        made = []
        base, out, fill = _beside(base, out, (T, N), x, M, rows, made)
        _check_like("out", out, x.dtype, (T, N))
        keep = u is not None and u is not False
        if u is True:
            u = _empty((M, R), torch.float32, x)
            made.append(u)
        elif not keep:
            u = None
        _check_like("u", u, torch.float32, (M, R))
        if ws is None:
            n = _sizes(lora_workspace_size, dev, dt, e, M, H, N, R)
            ws = _empty((n,), torch.uint8, x) if n else None
        call = lib().moe_lora_filled if fill else lib().moe_lora
        st = call(_dp(x), _dp(base), dt, T, _dp(a), _dp(b), _dp(scale), _dp(offsets), _dp(rows), e, M, H, N, R, _dp(out),
                  _dp(u), _dp(ws), _nbytes(ws), _current(dev))
    _check(st, "moe_lora")
    _hand_over(stream, *made)
    return (out, u) if keep else out


def lora_bwd(dout, x, u, a, b, offsets, rows=None, scale=None, base=None, need_dx=True, need_da=True, need_db=True,
             dx=None, da=None, db=None, dw_dtype=None, ws=None, stream=None):
    """moe_lora_bwd: the gradients of lora: dx (T,H), added to base where that is given
    (the shared projection's own gradient of x), da (e,H,R) and db (e,R,N), in x's type
    or float32 (dw_dtype). u: what lora kept. need_* False leaves one out (None).
    Returns (dx, da, db)."""
    T, N = dout.shape
    dev = dout.get_device()
    dt = _layer_dtype(dout)
    with _launch_on(dout, stream, x, u, a, b, offsets, rows, scale, base, dx, da, db, ws):
        e, M, H, N, R = _lora_shapes(T, N, "dout", a, b, offsets, rows, scale)
        _check_like("dout", dout, a.dtype, (T, N))
        _check_like("x", x, a.dtype, (T, H))
        _check_like("u", u, torch.float32, (M, R))
        made = []
        if need_dx:
            base, dx, fill = _beside(base, dx, (T, H), dout, M, rows, made)
        else:
            base, dx, fill = None, None, False
        wt = dw_dtype or a.dtype
        if not need_da:
            da = None
        elif da is None:
            da = _empty((e, H, R), wt, a)
            made.append(da)
        if not need_db:
            db = None
        elif db is None:
            db = _empty((e, R, N), wt, a)
            made.append(db)
        _check_like("dx", dx, dout.dtype, (T, H))
        given = da if da is not None else db
        wt = given.dtype if given is not None else wt
        _check_like("da", da, wt, (e, H, R))
        _check_like("db", db, wt, (e, R, N))
        if ws is None:
            n = _sizes(lora_bwd_workspace_size, dev, dt, e, M, H, N, R)
            ws = _empty((n,), torch.uint8, dout) if n else None
        call = lib().moe_lora_bwd_filled if fill else lib().moe_lora_bwd
        st = call(_dp(dout), _dp(x), _dp(u), dt, T, _dp(a), _dp(b), _dp(scale), _dp(offsets), _dp(rows), e, M, H, N, R,
                  _dp(base), _dp(dx), _dp(da), _dp(db), _CODE.get(wt, -1), _dp(ws), _nbytes(ws), _current(dev))
    _check(st, "moe_lora_bwd")
    _hand_over(stream, *made)
    return dx, da, db


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
