"""ctypes binding of the C ABI in include/moe.h (argument marshalling only).

Every function here has the name of the C entry point it calls and does no arithmetic of its
own: it checks dtypes/shapes of torch tensors, passes their device pointers and the current
CUDA stream, and turns a nonzero moe_status_t into an exception.  If the CUDA library is
missing, loading fails loudly; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_WORKSPACE = range(5)
MOE_DEV_BAD_EXPERT_ID, MOE_DEV_BAD_TOKEN_ID, MOE_DEV_NONFINITE, MOE_DEV_TIMEOUT = 1, 2, 4, 8
MOE_DEV_BAD_ADAPTER_ID = 16
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID, MOE_SCORE_HASH, MOE_SCORE_SQRTSOFTPLUS = 0, 1, 2, 3
MOE_SCORE_SOFTMAX_BIAS, MOE_SCORE_HASH_SQRTSOFTPLUS = 4, 5
MOE_FMT_NVFP4, MOE_FMT_MXFP4 = 0, 1
MOE_ACT_BF16, MOE_ACT_NVFP4 = 0, 1
MOE_DT_BF16, MOE_DT_F16 = 0, 1
MOE_FUNC_NONE, MOE_FUNC_SILU, MOE_FUNC_GELU, MOE_FUNC_GELU_TANH, MOE_FUNC_RELU = range(5)

# Every symbol include/moe.h declares.
EXPORTED = ["moe_route", "moe_workspace_size", "moe_prepare_weights", "moe_release_weights",
            "moe_ffn_forward", "moe_forward", "moe_workspace_size_host", "moe_forward_host",
            "moe_ffn_forward_noalloc", "moe_quantize_act_nvfp4", "moe_route_grouped", "moe_linear",
            "moe_add_rms_norm", "moe_linear_adapters", "moe_adapter_workspace_size", "moe_sandwich_norm",
            "moe_set_wait_limit", "moe_skew_barrier", "moe_profile_enable", "moe_profile_read",
            "moe_status_string"]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {moe_status_string(status)} (status {status})")
        self.status = status


class moe_qtensor(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("globals", ctypes.c_void_p), ("fmt", ctypes.c_int32)]


class moe_ffn_desc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("I_shared", ctypes.c_int32),
                ("gate", moe_qtensor), ("up", moe_qtensor), ("down", moe_qtensor),
                ("sh_gate", moe_qtensor), ("sh_up", moe_qtensor), ("sh_down", moe_qtensor),
                ("zero_experts", ctypes.c_int32)]


class moe_route_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("H", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("scoring", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("routed_scaling", ctypes.c_float),
                ("w_router", ctypes.c_void_p), ("correction_bias", ctypes.c_void_p),
                ("tid2eid", ctypes.c_void_p), ("vocab", ctypes.c_int64),
                ("token_ids", ctypes.c_void_p), ("zero_experts", ctypes.c_int32)]


class moe_linear_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("func", ctypes.c_int32), ("ldx", ctypes.c_int64),
                ("ldw", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldo", ctypes.c_int64)]


class moe_norm_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64),
                ("lds", ctypes.c_int64), ("ldo", ctypes.c_int64)]


class moe_adapter_desc(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int32), ("R", ctypes.c_int32), ("lda", ctypes.c_int64),
                ("sa", ctypes.c_int64), ("ldb", ctypes.c_int64), ("sb", ctypes.c_int64),
                ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("a_mul", ctypes.c_void_p),
                ("b_mul", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ids", ctypes.c_void_p)]


class moe_sandwich_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("wide", ctypes.c_int32), ("row_sigmoid", ctypes.c_int32), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("lds", ctypes.c_int64),
                ("ldo", ctypes.c_int64)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmoe_gb300.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_route.argtypes = [ctypes.POINTER(moe_route_desc), vp, vp, vp, vp, vp, vp, vp]
    lib.moe_route.restype = ctypes.c_int
    lib.moe_route_grouped.argtypes = [ctypes.POINTER(moe_route_desc), i32, i32, i32, vp, vp, vp, vp,
                                      vp, vp, vp]
    lib.moe_route_grouped.restype = ctypes.c_int
    lib.moe_linear.argtypes = [ctypes.POINTER(moe_linear_desc), vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_linear.restype = ctypes.c_int
    lib.moe_add_rms_norm.argtypes = [ctypes.POINTER(moe_norm_desc), vp, vp, vp, vp, vp, vp]
    lib.moe_add_rms_norm.restype = ctypes.c_int
    lib.moe_linear_adapters.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]  # descriptors as bytes, or by reference
    lib.moe_linear_adapters.restype = ctypes.c_int
    lib.moe_adapter_workspace_size.argtypes = [i32, i32, i32, ctypes.POINTER(sz)]
    lib.moe_adapter_workspace_size.restype = ctypes.c_int
    lib.moe_sandwich_norm.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_sandwich_norm.restype = ctypes.c_int
    lib.moe_workspace_size.argtypes = [ctypes.POINTER(moe_ffn_desc), i32, i32, ctypes.POINTER(sz)]
    lib.moe_workspace_size.restype = ctypes.c_int
    lib.moe_prepare_weights.argtypes = [ctypes.POINTER(moe_ffn_desc), ctypes.POINTER(vp), vp]
    lib.moe_prepare_weights.restype = ctypes.c_int
    lib.moe_release_weights.argtypes = [vp]
    lib.moe_release_weights.restype = ctypes.c_int
    lib.moe_ffn_forward.argtypes = [vp, i32, i32, f32, f32, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.moe_ffn_forward.restype = ctypes.c_int
    lib.moe_forward.argtypes = [vp, ctypes.POINTER(moe_route_desc), i32, f32, f32, vp, vp, vp, vp,
                                vp, vp, vp, sz, vp, vp]
    lib.moe_forward.restype = ctypes.c_int
    lib.moe_workspace_size_host.argtypes = [ctypes.POINTER(moe_ffn_desc), i32, i32, ctypes.POINTER(sz)]
    lib.moe_workspace_size_host.restype = ctypes.c_int
    lib.moe_forward_host.argtypes = [vp, ctypes.POINTER(moe_route_desc), i32, f32, f32, vp, vp, vp,
                                     vp, vp, vp, sz, vp, vp]
    lib.moe_forward_host.restype = ctypes.c_int
    lib.moe_ffn_forward_noalloc.argtypes = [vp, i32, i32, f32, f32, vp, vp, vp, vp, vp, vp]
    lib.moe_ffn_forward_noalloc.restype = ctypes.c_int
    lib.moe_quantize_act_nvfp4.argtypes = [vp, i64, i64, f32, vp, vp, vp]
    lib.moe_quantize_act_nvfp4.restype = ctypes.c_int
    lib.moe_set_wait_limit.argtypes = [vp, ctypes.c_uint64]
    lib.moe_set_wait_limit.restype = ctypes.c_int
    lib.moe_skew_barrier.argtypes = [vp, vp]
    lib.moe_skew_barrier.restype = ctypes.c_int
    lib.moe_profile_enable.argtypes = [vp, ctypes.c_uint32]
    lib.moe_profile_enable.restype = ctypes.c_int
    lib.moe_profile_read.argtypes = [vp, ctypes.POINTER(ctypes.c_float)]
    lib.moe_profile_read.restype = ctypes.c_int
    _lib = lib
    return lib


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _dptr(t: Optional[torch.Tensor], dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _hptr(t: Optional[torch.Tensor], dtype, name="tensor"):
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


_DTYPES = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}


def _stream_device(stream):
    """The stream's handle and the current device, which every tensor of the call must be on."""
    dev = torch.cuda.current_device()
    if stream is None:  # the handle alone: a Stream object costs 3 us of host time
        return torch._C._cuda_getCurrentRawStream(dev), dev
    if stream.device_index != dev:
        raise ValueError("the stream must belong to the current CUDA device")
    return stream.cuda_stream, dev


def _tptr(t, dtype, shape, dev, name):
    """Pointer of a contiguous tensor of a stated type and shape on the current device."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on the current CUDA "
                         f"device, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t, dtype, rows, cols, dev, name):
    """Pointer and row stride of a matrix of a stated type whose rows are contiguous."""
    if t.dtype != dtype or t.shape != (rows, cols) or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} matrix {(rows, cols)} on the current CUDA device, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), (ld if rows > 1 else cols)


def qtensor(p: Optional[dict]) -> moe_qtensor:
    """Weight dict {packed, scales, globals, fmt} of CUDA tensors -> moe_qtensor."""
    if p is None:
        return moe_qtensor(None, None, None, 0)
    return moe_qtensor(_dptr(p["packed"], torch.uint8, "packed"),
                       _dptr(p["scales"], torch.uint8, "scales"),
                       _dptr(p.get("globals"), torch.float32, "globals"), int(p["fmt"]))


def ffn_desc(E, H, I, top_k, I_shared, gate, up, down, sh_gate=None, sh_up=None, sh_down=None,
             zero_experts=0):
    return moe_ffn_desc(E, H, I, top_k, I_shared, qtensor(gate), qtensor(up), qtensor(down),
                        qtensor(sh_gate), qtensor(sh_up), qtensor(sh_down), int(zero_experts))


def route_desc(*, T, E, H, top_k, scoring, renormalize, routed_scaling, w_router=None,
               correction_bias=None, tid2eid=None, vocab=0, token_ids=None,
               zero_experts=0) -> moe_route_desc:
    return moe_route_desc(int(T), int(E), int(H), int(top_k), int(scoring), int(bool(renormalize)),
                          float(routed_scaling), _dptr(w_router, torch.bfloat16, "w_router"),
                          _dptr(correction_bias, torch.float32, "correction_bias"),
                          _dptr(tid2eid, torch.int64, "tid2eid"), int(vocab),
                          _dptr(token_ids, torch.int32, "token_ids"), int(zero_experts))


def moe_route(*, T, E, H, top_k, scoring, renormalize, routed_scaling, x=None, w_router=None,
              logits_in=None, logits_out=None, correction_bias=None, tid2eid=None, vocab=0,
              token_ids=None, topk_ids, topk_w, dev_status=None, stream=None, zero_experts=0):
    lib = load_library()
    d = route_desc(T=T, E=E, H=H, top_k=top_k, scoring=scoring, renormalize=renormalize,
                   routed_scaling=routed_scaling, w_router=w_router,
                   correction_bias=correction_bias, tid2eid=tid2eid, vocab=vocab,
                   token_ids=token_ids, zero_experts=zero_experts)
    st = lib.moe_route(ctypes.byref(d), _dptr(x, torch.bfloat16, "x"),
                       _dptr(logits_in, torch.float32, "logits_in"),
                       _dptr(logits_out, torch.float32, "logits_out"),
                       _dptr(topk_ids, torch.int32, "topk_ids"), _dptr(topk_w, torch.float32, "topk_w"),
                       _dptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "moe_route")


def moe_route_grouped(*, T, E, H, top_k, scoring, renormalize, routed_scaling, n_group, topk_group,
                      group_top=1, x=None, w_router=None, logits_in=None, logits_out=None,
                      correction_bias=None, topk_ids, topk_w, dev_status=None, stream=None):
    """moe_route with the top-K limited to the topk_group best of n_group expert groups."""
    st, dev = _stream_device(stream)
    E, H, top_k, T = int(E), int(H), int(top_k), int(T)
    given = logits_in is not None
    d = moe_route_desc(T, E, H, top_k, scoring, 1 if renormalize else 0, routed_scaling,
                       None if given else _tptr(w_router, torch.bfloat16, (E, H), dev, "w_router"),
                       _tptr(correction_bias, torch.float32, (E,), dev, "correction_bias"),
                       None, 0, None, 0)
    rc = (_lib or load_library()).moe_route_grouped(
        ctypes.byref(d), n_group, topk_group, group_top,
        None if given else _tptr(x, torch.bfloat16, (T, H), dev, "x"),
        _tptr(logits_in, torch.float32, (T, E), dev, "logits_in"),
        _tptr(logits_out, torch.float32, (T, E), dev, "logits_out"),
        _tptr(topk_ids, torch.int32, (T, top_k), dev, "topk_ids"),
        _tptr(topk_w, torch.float32, (T, top_k), dev, "topk_w"),
        _tptr(dev_status, torch.int32, (1,), dev, "dev_status"), st)
    if rc != MOE_OK:
        raise MoeError(rc, "moe_route_grouped")


def moe_linear(x, w, out, *, w_mul=None, bias=None, bias_mul=None, residual=None, func=MOE_FUNC_NONE,
               dev_status=None, stream=None):
    """out = f(x w^T + bias) [* (x w_mul^T + bias_mul)] [+ residual]; x [T][K], w and w_mul [N][K],
    residual and out [T][N] of one type (bf16 or f16), rows of any stride."""
    st, dev = _stream_device(stream)
    dt = x.dtype
    T, K = x.shape
    N = w.shape[0]
    px, ldx = _rows(x, dt, T, K, dev, "x")
    pw, ldw = _rows(w, dt, N, K, dev, "w")
    po, ldo = _rows(out, dt, T, N, dev, "out")
    pm = pr = None
    ldr = N
    if w_mul is not None:
        pm, ldm = _rows(w_mul, dt, N, K, dev, "w_mul")
        if ldm != ldw:
            raise ValueError("w_mul must have the row stride of w")
    if residual is not None:
        pr, ldr = _rows(residual, dt, T, N, dev, "residual")
    d = moe_linear_desc(T, N, K, _DTYPES.get(dt, -1), func, ldx, ldw, ldr, ldo)
    rc = (_lib or load_library()).moe_linear(
        ctypes.byref(d), px, pw, pm, _tptr(bias, torch.float32, (N,), dev, "bias"),
        _tptr(bias_mul, torch.float32, (N,), dev, "bias_mul"), pr, po,
        _tptr(dev_status, torch.int32, (1,), dev, "dev_status"), st)
    if rc != MOE_OK:
        raise MoeError(rc, "moe_linear")


def moe_add_rms_norm(x, weight, out, *, residual=None, sum_out=None, eps=1e-6, stream=None):
    """s = x + residual; out = s * weight / sqrt(mean(s^2) + eps); sum_out = s.  x, residual, sum_out
    and out [T][H], weight [H], of one type (bf16 or f16), rows of any stride."""
    st, dev = _stream_device(stream)
    dt = x.dtype
    T, H = x.shape
    px, ldx = _rows(x, dt, T, H, dev, "x")
    po, ldo = _rows(out, dt, T, H, dev, "out")
    pr = ps = None
    ldr = lds = H
    if residual is not None:
        pr, ldr = _rows(residual, dt, T, H, dev, "residual")
    if sum_out is not None:
        ps, lds = _rows(sum_out, dt, T, H, dev, "sum_out")
    d = moe_norm_desc(T, H, _DTYPES.get(dt, -1), eps, ldx, ldr, lds, ldo)
    rc = (_lib or load_library()).moe_add_rms_norm(ctypes.byref(d), px, pr, _tptr(weight, dt, (H,), dev, "weight"),
                                         ps, po, st)
    if rc != MOE_OK:
        raise MoeError(rc, "moe_add_rms_norm")


# The descriptors of the two calls below as bytes, in the order of the structures' fields: a ctypes structure of
# as many costs 1 us of host time.
_LINEAR = struct.Struct("5i4x4q")
_ADAPTER = struct.Struct("2i4q6P")
_SANDWICH = struct.Struct("5i3f4q")
assert _LINEAR.size == ctypes.sizeof(moe_linear_desc) and _ADAPTER.size == ctypes.sizeof(moe_adapter_desc)
assert _SANDWICH.size == ctypes.sizeof(moe_sandwich_desc)


def _stack(t, dtype, L, rows, cols, dev, name):
    """Pointer, row and adapter stride of stacked adapter matrices [L][rows][cols]."""
    if t.dtype != dtype or t.shape != (L, rows, cols) or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor {(L, rows, cols)} on the current CUDA device, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    step, ld, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} must have contiguous rows")
    ld = ld if rows > 1 else cols
    return t.data_ptr(), ld, (step if L > 1 else rows * ld)  # a lone adapter has no distance


def _pair(a, b, dtype, L, R, N, K, dev, name):
    """Pointers and strides of the adapters of one matrix, zeros without any."""
    if a is None and b is None:
        return 0, 0, None
    if a is None or b is None:
        raise ValueError(f"adapters need a{name} and b{name}")
    pa, lda, sa = _stack(a, dtype, L, R, K, dev, "a" + name)
    pb, ldb, sb = _stack(b, dtype, L, N, R, dev, "b" + name)
    return pa, pb, (lda, sa, ldb, sb)


def moe_adapter_workspace_size(T: int, R: int, matrices: int) -> int:
    n = ctypes.c_size_t(0)
    rc = (_lib or load_library()).moe_adapter_workspace_size(T, R, matrices, ctypes.byref(n))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_adapter_workspace_size")
    return n.value


def moe_linear_adapters(x, w, out, ids, *, a=None, b=None, a_mul=None, b_mul=None, scale=None, w_mul=None,
                        bias=None, bias_mul=None, residual=None, func=MOE_FUNC_NONE, workspace,
                        dev_status=None, stream=None):
    """moe_linear with low-rank adapters: x w^T gains scale[j] (x a[j]^T) b[j]^T for the adapter j = ids[t] of
    each row (-1: none), x w_mul^T the same of a_mul and b_mul.  ids int32 [T]; a and a_mul [L][R][K], b and b_mul
    [L][N][R], of the layer's type; scale float [L]; workspace: moe_adapter_workspace_size(T, R, matrices) bytes."""
    st, dev = _stream_device(stream)
    dt = x.dtype
    T, K = x.shape
    N = w.shape[0]
    first = a if a is not None else a_mul
    if first is None or first.dim() != 3:
        raise ValueError("adapters must be given as a and b, or a_mul and b_mul, of three dimensions")
    L, R, _ = first.shape
    px, ldx = _rows(x, dt, T, K, dev, "x")
    pw, ldw = _rows(w, dt, N, K, dev, "w")
    po, ldo = _rows(out, dt, T, N, dev, "out")
    pm = pr = None
    ldr = N
    if w_mul is not None:
        pm, ldm = _rows(w_mul, dt, N, K, dev, "w_mul")
        if ldm != ldw:
            raise ValueError("w_mul must have the row stride of w")
    if residual is not None:
        pr, ldr = _rows(residual, dt, T, N, dev, "residual")
    pa, pb, strides = _pair(a, b, dt, L, R, N, K, dev, "")
    pa_mul, pb_mul, strides_mul = _pair(a_mul, b_mul, dt, L, R, N, K, dev, "_mul")
    if strides is None:
        strides = strides_mul
    elif strides_mul is not None and strides != strides_mul:
        raise ValueError("a_mul and b_mul must have the strides of a and b")
    if workspace.dtype != torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the current CUDA device")
    if max(L, R, N, K, T) > 0x7FFFFFFF:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_linear_adapters")
    rc = (_lib or load_library()).moe_linear_adapters(
        _LINEAR.pack(T, N, K, _DTYPES.get(dt, -1), func, ldx, ldw, ldr, ldo),
        _ADAPTER.pack(L, R, *strides, pa, pb, pa_mul, pb_mul, _tptr(scale, torch.float32, (L,), dev, "scale") or 0,
                      _tptr(ids, torch.int32, (T,), dev, "ids") or 0),
        px, pw, pm, None if bias is None else _tptr(bias, torch.float32, (N,), dev, "bias"),
        None if bias_mul is None else _tptr(bias_mul, torch.float32, (N,), dev, "bias_mul"), pr, po, workspace.data_ptr(),
        workspace.numel(), None if dev_status is None else _tptr(dev_status, torch.int32, (1,), dev, "dev_status"), st)
    if rc != MOE_OK:
        raise MoeError(rc, "moe_linear_adapters")


def moe_sandwich_norm(x, sum_out, *, residual=None, post_weight=None, gate=None, row_gate=None, row_sigmoid=False,
                      weight=None, out=None, residual_scale=1.0, weight_offset=0.0, eps=1e-6, stream=None):
    """p = norm(x) * (post_weight + weight_offset), or x without post_weight; sum_out = residual_scale * residual +
    row_gate * gate * p; out = norm(sum) * (weight + weight_offset).  x and out [T][H], post_weight, gate and weight [H]
    of one type (bf16 or f16); residual and sum_out [T][H] of that type or float32; row_gate float32 [T], with
    row_sigmoid its logits; rows of any stride."""
    st, dev = _stream_device(stream)
    dt = x.dtype
    T, H = x.shape
    stream_dt = sum_out.dtype
    if stream_dt != dt and stream_dt != torch.float32:
        raise ValueError(f"sum_out must be of the type of x or float32, got {stream_dt}")
    px, ldx = _rows(x, dt, T, H, dev, "x")
    ps, lds = _rows(sum_out, stream_dt, T, H, dev, "sum_out")
    pr = po = None
    ldr = ldo = H
    if residual is not None:
        pr, ldr = _rows(residual, stream_dt, T, H, dev, "residual")
    if out is not None:
        po, ldo = _rows(out, dt, T, H, dev, "out")
    if max(T, H) > 0x7FFFFFFF:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_sandwich_norm")
    rc = (_lib or load_library()).moe_sandwich_norm(
        _SANDWICH.pack(T, H, _DTYPES.get(dt, -1), stream_dt == torch.float32, bool(row_sigmoid), eps, residual_scale,
                       weight_offset, ldx, ldr, lds, ldo),
        px, pr, None if post_weight is None else _tptr(post_weight, dt, (H,), dev, "post_weight"),
        None if gate is None else _tptr(gate, dt, (H,), dev, "gate"),
        None if row_gate is None else _tptr(row_gate, torch.float32, (T,), dev, "row_gate"),
        None if weight is None else _tptr(weight, dt, (H,), dev, "weight"), ps, po, st)
    if rc != MOE_OK:
        raise MoeError(rc, "moe_sandwich_norm")


def moe_workspace_size(desc: moe_ffn_desc, T: int, act: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_workspace_size(ctypes.byref(desc), int(T), int(act), ctypes.byref(n)),
           "moe_workspace_size")
    return int(n.value)


def moe_prepare_weights(desc: moe_ffn_desc, stream=None) -> int:
    h = ctypes.c_void_p(None)
    _check(load_library().moe_prepare_weights(ctypes.byref(desc), ctypes.byref(h), _stream(stream)),
           "moe_prepare_weights")
    return h.value


def moe_release_weights(handle: int):
    _check(load_library().moe_release_weights(ctypes.c_void_p(handle)), "moe_release_weights")


def moe_ffn_forward(handle: int, T: int, act: int, g_act1: float, g_act2: float, x, topk_ids,
                    topk_w, out, workspace, dev_status=None, stream=None):
    st = load_library().moe_ffn_forward(
        ctypes.c_void_p(handle), int(T), int(act), float(g_act1), float(g_act2),
        _dptr(x, torch.bfloat16, "x"), _dptr(topk_ids, torch.int32, "topk_ids"),
        _dptr(topk_w, torch.float32, "topk_w"), _dptr(out, torch.bfloat16, "out"),
        _dptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _dptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "moe_ffn_forward")


def moe_forward(handle: int, route: moe_route_desc, act: int, g_act1: float, g_act2: float, x,
                topk_ids, topk_w, out, workspace, logits_in=None, logits_out=None,
                dev_status=None, stream=None):
    """Route + expert FFN in one call (one persistent launch for a few tokens)."""
    st = load_library().moe_forward(
        ctypes.c_void_p(handle), ctypes.byref(route), int(act), float(g_act1), float(g_act2),
        _dptr(x, torch.bfloat16, "x"), _dptr(logits_in, torch.float32, "logits_in"),
        _dptr(logits_out, torch.float32, "logits_out"), _dptr(topk_ids, torch.int32, "topk_ids"),
        _dptr(topk_w, torch.float32, "topk_w"), _dptr(out, torch.bfloat16, "out"),
        _dptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _dptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "moe_forward")


def moe_workspace_size_host(desc: moe_ffn_desc, T: int, act: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_workspace_size_host(ctypes.byref(desc), int(T), int(act),
                                                  ctypes.byref(n)), "moe_workspace_size_host")
    return int(n.value)


def moe_forward_host(handle: int, route: moe_route_desc, act: int, g_act1: float, g_act2: float,
                     x_host, out_host, workspace, token_ids_host=None, topk_ids_host=None,
                     topk_w_host=None, dev_status=None, stream=None):
    """moe_forward on host buffers (CPU tensors, pinned for asynchronous copies): the copies in
    and out are enqueued on the stream with the forward; synchronise before reading out_host."""
    st = load_library().moe_forward_host(
        ctypes.c_void_p(handle), ctypes.byref(route), int(act), float(g_act1), float(g_act2),
        _hptr(x_host, torch.bfloat16, "x_host"), _hptr(token_ids_host, torch.int32, "token_ids_host"),
        _hptr(out_host, torch.bfloat16, "out_host"), _hptr(topk_ids_host, torch.int32, "topk_ids_host"),
        _hptr(topk_w_host, torch.float32, "topk_w_host"),
        _dptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _dptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "moe_forward_host")


def moe_ffn_forward_noalloc(handle: int, T: int, act: int, g_act1: float, g_act2: float, x,
                            topk_ids, topk_w, out, dev_status=None, stream=None):
    """moe_ffn_forward with the library's static device workspace (no caller allocation)."""
    st = load_library().moe_ffn_forward_noalloc(
        ctypes.c_void_p(handle), int(T), int(act), float(g_act1), float(g_act2),
        _dptr(x, torch.bfloat16, "x"), _dptr(topk_ids, torch.int32, "topk_ids"),
        _dptr(topk_w, torch.float32, "topk_w"), _dptr(out, torch.bfloat16, "out"),
        _dptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "moe_ffn_forward_noalloc")


def moe_quantize_act_nvfp4(x, g: float, packed, scales, stream=None):
    rows, K = x.shape
    st = load_library().moe_quantize_act_nvfp4(
        _dptr(x, torch.bfloat16, "x"), int(rows), int(K), float(g),
        _dptr(packed, torch.uint8, "packed"), _dptr(scales, torch.uint8, "scales"), _stream(stream))
    _check(st, "moe_quantize_act_nvfp4")


def moe_set_wait_limit(handle: int, cycles: int):
    _check(load_library().moe_set_wait_limit(ctypes.c_void_p(handle), int(cycles)),
           "moe_set_wait_limit")


def moe_skew_barrier(handle: int, stream=None):
    _check(load_library().moe_skew_barrier(ctypes.c_void_p(handle), _stream(stream)),
           "moe_skew_barrier")


PHASE_DISPATCH, PHASE_GATE_UP, PHASE_DOWN, PHASE_COMBINE = 0, 1, 2, 3


def moe_profile_enable(handle: int, mask: int):
    _check(load_library().moe_profile_enable(ctypes.c_void_p(handle), int(mask)), "moe_profile_enable")


def moe_profile_read(handle: int):
    ms = (ctypes.c_float * 4)()
    _check(load_library().moe_profile_read(ctypes.c_void_p(handle), ms), "moe_profile_read")
    return [float(v) for v in ms]
