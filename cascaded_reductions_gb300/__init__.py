"""cascaded_reductions_gb300 -- Python binding of librf.so.

Argument marshalling only: every step of every cascade runs in the library's
CUDA kernels.  Each ``rf_*`` function here has the name and meaning of the C
entry point declared in ``include/rf.h``; it takes torch CUDA tensors, checks
their dtype, shape and contiguity, and passes raw device pointers and the
current stream.  A status other than RF_OK raises :class:`RFError`.

The convenience wrappers (``attn_decode``, ``softmax_topk``,
``absmax_quant_fp8_gemm``, ``attn_prefill``) only allocate the output tensors
with torch and call the entry points; so do ``attn_prefill_window``,
``attn_decode_window``, ``attn_decode_shared``, ``attn_decode_weights`` and
``cache_evict``, which work over a serving cache of grouped heads, with scratch
from ``decode_workspace`` where a loop keeps it.

There is no fallback: importing this package fails if librf.so has not been
built (``cascaded_reductions_gb300._build.build()``).  The environment
variable ``RF_LIBRARY`` names another build of the same library to load
instead, e.g. the bounds-checked debug variant that
``cascaded_reductions_gb300._build.build_checked()`` makes.
"""

import ctypes
import os
import typing
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("RF_LIBRARY") or os.path.join(_HERE, "librf.so")

(RF_OK, RF_ERR_INVALID_ARG, RF_ERR_UNSUPPORTED, RF_ERR_MISALIGNED, RF_ERR_CUDA, RF_ERR_TIMEOUT,
 RF_ERR_BOUNDS) = range(7)
RF_F32, RF_BF16, RF_F16 = 0, 1, 2
RF_FUSE_NONE, RF_FUSE_THREAD, RF_FUSE_WARP, RF_FUSE_BLOCK = range(4)

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float

_SIGNATURES = {
    "rf_status_string": (ctypes.c_char_p, [_I]),
    "rf_version": (_I, []),
    "rf_attn_decode_split": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P]),
    "rf_state_merge": (_I, [_P, _P, _P, _I, _I, _I, _P, _I, _P, _P]),
    "rf_attn_prefill": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "rf_softmax_topk": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
    "rf_absmax_quant_fp8_gemm": (_I, [_P, _I, _I, _P, _P, _I, _P, _P, _P, _P]),
    "rf_absmax_quant_e4m3": (_I, [_P, _I, _I, _P, _P, _P]),
    "rf_fp8_gemm_scaled": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "rf_device_error": (_I, [ctypes.POINTER(_I), _P]),
    "rf_attn_decode_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _I, _P, _P]),
    "rf_row_softmax": (_I, [_P, _I, _I, _P, _I, _P, _P]),
    "rf_row_variance": (_I, [_P, _I, _I, _P, _P, _I, _P]),
    "rf_moment_of_inertia": (_I, [_P, _P, _I, _I, _P, _P, _I, _P]),
    "rf_layer_norm": (_I, [_P, _P, _P, _I, _I, _F, _P, _I, _P, _P]),
    "rf_attn_decode_split_twopass": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P]),
    "rf_incremental_quant_fp8_gemm": (_I, [_P, _I, _I, _P, _P, _I, _P, _P, _P]),
    "rf_mla_decode_split": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P]),
    "rf_selftest_wait_timeout": (_I, [_P, _P]),
    "rf_rms_norm": (_I, [_P, _P, _I, _I, _F, _P, _I, _P, _P]),
    "rf_attn_decode_fused": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P, _P, _I, _P, _P]),
    "rf_bounds_checked": (_I, []),
    "rf_selftest_bounds": (_I, [_P]),
    "rf_stream_read": (_I, [_P, ctypes.c_size_t, _P, _P]),
    "rf_decode_segments": (_I, [_I, _I]),
    "rf_attn_decode_window": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P,
                                   _P, _P, _P, _I, _P, _P]),
    "rf_attn_decode_weights": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P,
                                    _P, _P, _I, _P, _P, _P, _P]),
    "rf_attn_prefill_window": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P,
                                    _P]),
    "rf_prefix_segments": (_I, [_I, _I, _I, _I]),
    "rf_attn_decode_shared": (_I, [_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I,
                                   _P, _P, _P, _P, _P, _I, _P, _P]),
    "rf_cache_evict": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P,
                            _P]),
}


def load_library(path=LIB_PATH):
    """Open librf.so and declare every entry point's C signature."""
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run cascaded_reductions_gb300._build.build() "
            "(nvcc for sm_103a).  There is no CPU fallback.")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = load_library()


def _load_calls():
    """The extension built from csrc/calls.cpp, or None where it is not there or does not load (with
    a warning): the wrappers below then marshal the same calls in Python."""
    from . import _build
    path, _ = _build.calls_path()
    if path is None or not os.path.exists(path):
        return None
    import importlib.machinery
    import importlib.util
    loader = importlib.machinery.ExtensionFileLoader("_rf_calls", path)
    try:
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_rf_calls", loader))
        loader.exec_module(module)
    except (ImportError, OSError) as e:
        warnings.warn(f"{os.path.basename(path)} does not load, its calls are marshalled in Python: {e}",
                      RuntimeWarning, stacklevel=2)
        return None
    return module


_calls = _load_calls()


def _entry(name):
    return ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value


(_DECODE_WINDOW, _PREFILL_WINDOW, _DECODE_SHARED, _DECODE_WEIGHTS, _CACHE_EVICT) = map(
    _entry, ("rf_attn_decode_window", "rf_attn_prefill_window", "rf_attn_decode_shared",
             "rf_attn_decode_weights", "rf_cache_evict"))


class RFError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {_lib.rf_status_string(status).decode()}")


def _check(status, where):
    if status != RF_OK:
        raise RFError(status, where)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t, dtype, name, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _dtype_code(dt):
    if dt == torch.float32:
        return RF_F32
    if dt == torch.bfloat16:
        return RF_BF16
    raise ValueError(f"unsupported dtype {dt}")


# The calls over a cache of grouped heads run on the device that holds their
# tensors, whichever is current: their arguments share one device, and the
# stream (by default that device's current one) belongs to it.

_CACHE_DTYPES = {torch.float32: RF_F32, torch.bfloat16: RF_BF16, torch.float16: RF_F16}


def _cache_dtype(dt, name):
    code = _CACHE_DTYPES.get(dt)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {dt}")
    return code


# the current stream's handle and the current device, without making objects of
# them: a decode step is a handful of microseconds
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device_of(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _on(dev, t, dtype, shape, name):
    """``t`` as it has to be: on device ``dev`` (an index), of a type and shape, contiguous."""
    if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return
    _need(t, dtype, name, shape)
    raise ValueError(f"{name} is on {t.device}, other tensors on cuda:{dev}: one call works on one device")


def _call_on(dev, stream, where, fn, *args):
    """fn(*args, stream) with device ``dev`` (an index) current; raises RFError on a bad status."""
    if stream is None:
        ptr = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream of {stream.device} for tensors on cuda:{dev}")
    else:
        ptr = stream.cuda_stream
    if _current_device() == dev:
        status = fn(*args, ptr)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, ptr)
    if status != RF_OK:
        raise RFError(status, where)


def _i32(n):
    """A count for a C int: one too large for it is as good as the largest."""
    return n if -1 <= n <= 0x7fffffff else (0x7fffffff if n > 0 else -1)


def _c_ints(*counts):
    """Counts for C ints (ctypes would cut off their high bits)."""
    return tuple(map(_i32, counts))


def _addr(t):
    """The address of an optional tensor: null for None, and only then."""
    if t is None:
        return None
    p = t.data_ptr()
    if p == 0 and t.numel() > 0:
        raise ValueError("a tensor without memory")
    return p


def version():
    return _lib.rf_version()


# ------------------------------------------------------------ entry points --

def rf_attn_decode_split(q, k, v, S, scale, seg_m, seg_l, seg_acc, stream=None):
    """q [R, D], k/v [R, L, D] (fp32 D=64 or bf16 D=128) -> seg_m/seg_l [R, S], seg_acc [R, S, D]."""
    R, L, D = k.shape
    _need(q, k.dtype, "q", (R, D))
    _need(k, k.dtype, "k")
    _need(v, k.dtype, "v", (R, L, D))
    _need(seg_m, torch.float32, "seg_m", (R, S))
    _need(seg_l, torch.float32, "seg_l", (R, S))
    _need(seg_acc, torch.float32, "seg_acc", (R, S, D))
    _check(_lib.rf_attn_decode_split(_ptr(q), _ptr(k), _ptr(v), R, L, D, S, float(scale),
                                     _dtype_code(k.dtype), _ptr(seg_m), _ptr(seg_l), _ptr(seg_acc),
                                     _stream(stream)), "rf_attn_decode_split")


def rf_attn_decode_fused(q, k, v, S, scale, seg_m, seg_l, seg_acc, counters, out, lse=None,
                         stream=None):
    """Split-KV decode with the merge done by each row's last CTA, in one launch.
    counters: int32 [R] CUDA tensor, zero before the first call (calls leave it zero)."""
    R, L, D = k.shape
    dt = _dtype_code(q.dtype)
    _need(q, q.dtype, "q", (R, D))
    _need(k, q.dtype, "k", (R, L, D))
    _need(v, q.dtype, "v", (R, L, D))
    _need(seg_m, torch.float32, "seg_m", (R, S))
    _need(seg_l, torch.float32, "seg_l", (R, S))
    _need(seg_acc, torch.float32, "seg_acc", (R, S, D))
    _need(counters, torch.int32, "counters", (R,))
    _need(out, out.dtype, "out", (R, D))
    if lse is not None:
        _need(lse, torch.float32, "lse", (R,))
    _check(_lib.rf_attn_decode_fused(_ptr(q), _ptr(k), _ptr(v), R, L, D, S, float(scale), dt,
                                     _ptr(seg_m), _ptr(seg_l), _ptr(seg_acc), _ptr(counters),
                                     _ptr(out), _dtype_code(out.dtype), _ptr(lse), _stream(stream)),
           "rf_attn_decode_fused")


def rf_attn_decode_split_twopass(q, k, v, S, scale, seg_m, seg_l, seg_acc, stream=None):
    """Non-incremental split-KV decode: same arguments and outputs as
    rf_attn_decode_split; segments of at most 16384 keys."""
    R, L, D = k.shape
    _need(q, k.dtype, "q", (R, D))
    _need(k, k.dtype, "k")
    _need(v, k.dtype, "v", (R, L, D))
    _need(seg_m, torch.float32, "seg_m", (R, S))
    _need(seg_l, torch.float32, "seg_l", (R, S))
    _need(seg_acc, torch.float32, "seg_acc", (R, S, D))
    _check(_lib.rf_attn_decode_split_twopass(_ptr(q), _ptr(k), _ptr(v), R, L, D, S, float(scale),
                                             _dtype_code(k.dtype), _ptr(seg_m), _ptr(seg_l),
                                             _ptr(seg_acc), _stream(stream)),
           "rf_attn_decode_split_twopass")


def rf_mla_decode_split(q, c, S, scale, seg_m, seg_l, seg_acc, stream=None):
    """q [B, H, 576], c [B, L, 576] bf16 (shared latent cache) -> seg_m/seg_l [B, H, S],
    seg_acc [B, H, S, 512] fp32."""
    B, H, Dk = q.shape
    L = c.shape[1]
    Dv = seg_acc.shape[-1]
    _need(q, torch.bfloat16, "q")
    _need(c, torch.bfloat16, "c", (B, L, Dk))
    _need(seg_m, torch.float32, "seg_m", (B, H, S))
    _need(seg_l, torch.float32, "seg_l", (B, H, S))
    _need(seg_acc, torch.float32, "seg_acc", (B, H, S, Dv))
    _check(_lib.rf_mla_decode_split(_ptr(q), _ptr(c), B, H, L, Dk, Dv, S, float(scale),
                                    _ptr(seg_m), _ptr(seg_l), _ptr(seg_acc), _stream(stream)),
           "rf_mla_decode_split")


def rf_state_merge(seg_m, seg_l, seg_acc, out, lse=None, stream=None):
    """seg_* [R, S(, D)] fp32 -> out [R, D] (fp32 or bf16), lse [R] fp32 (optional)."""
    R, S, D = seg_acc.shape
    _need(seg_m, torch.float32, "seg_m", (R, S))
    _need(seg_l, torch.float32, "seg_l", (R, S))
    _need(seg_acc, torch.float32, "seg_acc")
    _need(out, out.dtype, "out", (R, D))
    if lse is not None:
        _need(lse, torch.float32, "lse", (R,))
    _check(_lib.rf_state_merge(_ptr(seg_m), _ptr(seg_l), _ptr(seg_acc), R, S, D, _ptr(out),
                               _dtype_code(out.dtype), _ptr(lse), _stream(stream)),
           "rf_state_merge")


def rf_attn_prefill(q, k, v, causal, scale, out, lse=None, stream=None):
    """q/k/v/out [B, H, N, D] bf16; lse [B, H, N] fp32 (optional)."""
    B, H, N, D = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _need(t, torch.bfloat16, name, (B, H, N, D))
    if lse is not None:
        _need(lse, torch.float32, "lse", (B, H, N))
    _check(_lib.rf_attn_prefill(_ptr(q), _ptr(k), _ptr(v), B, H, N, D, int(bool(causal)),
                                float(scale), _ptr(out), _ptr(lse), _stream(stream)),
           "rf_attn_prefill")


def rf_softmax_topk(logits, k, renormalize, idx, w, stream=None):
    """logits [T, E] fp32 -> idx [T, k] int32, w [T, k] fp32."""
    T, E = logits.shape
    _need(logits, torch.float32, "logits")
    _need(idx, torch.int32, "idx", (T, k))
    _need(w, torch.float32, "w", (T, k))
    _check(_lib.rf_softmax_topk(_ptr(logits), T, E, k, int(bool(renormalize)), _ptr(idx), _ptr(w),
                                _stream(stream)), "rf_softmax_topk")


def rf_absmax_quant_e4m3(x, xq, sx, stream=None):
    """x [M, K] bf16 -> xq [M, K] uint8 (e4m3 codes), sx [M] fp32."""
    M, K = x.shape
    _need(x, torch.bfloat16, "x")
    _need(xq, torch.uint8, "xq", (M, K))
    _need(sx, torch.float32, "sx", (M,))
    _check(_lib.rf_absmax_quant_e4m3(_ptr(x), M, K, _ptr(xq), _ptr(sx), _stream(stream)),
           "rf_absmax_quant_e4m3")


def rf_fp8_gemm_scaled(xq, sx, wq, sw, y, stream=None):
    """xq [M, K], wq [N, K] uint8 e4m3; sx [M], sw [N] fp32 -> y [M, N] bf16."""
    M, K = xq.shape
    N = wq.shape[0]
    _need(xq, torch.uint8, "xq")
    _need(wq, torch.uint8, "wq", (N, K))
    _need(sx, torch.float32, "sx", (M,))
    _need(sw, torch.float32, "sw", (N,))
    _need(y, torch.bfloat16, "y", (M, N))
    _check(_lib.rf_fp8_gemm_scaled(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), M, N, K, _ptr(y),
                                   _stream(stream)), "rf_fp8_gemm_scaled")


def rf_absmax_quant_fp8_gemm(x, wq, sw, xq, sx, y, stream=None):
    """x [M, K] bf16, wq [N, K] uint8, sw [N] -> xq [M, K] uint8, sx [M], y [M, N] bf16."""
    M, K = x.shape
    N = wq.shape[0]
    _need(x, torch.bfloat16, "x")
    _need(wq, torch.uint8, "wq", (N, K))
    _need(sw, torch.float32, "sw", (N,))
    _need(xq, torch.uint8, "xq", (M, K))
    _need(sx, torch.float32, "sx", (M,))
    _need(y, torch.bfloat16, "y", (M, N))
    _check(_lib.rf_absmax_quant_fp8_gemm(_ptr(x), M, K, _ptr(wq), _ptr(sw), N, _ptr(xq), _ptr(sx),
                                         _ptr(y), _stream(stream)), "rf_absmax_quant_fp8_gemm")


def rf_attn_decode_noalloc(q, k, v, S, scale, out, lse=None, stream=None):
    """Decode split + merge with the segment states in the library's fixed
    16 MiB device array: for callers that cannot allocate device memory.

    q [R, D], k/v [R, L, D] (fp32 D=64 or bf16 D=128); out [R, D] fp32 or
    bf16; lse [R] fp32 (optional).  Calls that may overlap on the GPU share the
    array and race; the first call on a device must precede stream capture."""
    R, L, D = k.shape
    _need(q, k.dtype, "q", (R, D))
    _need(k, k.dtype, "k")
    _need(v, k.dtype, "v", (R, L, D))
    _need(out, out.dtype, "out", (R, D))
    if lse is not None:
        _need(lse, torch.float32, "lse", (R,))
    _check(_lib.rf_attn_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), R, L, D, S, float(scale),
                                       _dtype_code(k.dtype), _ptr(out), _dtype_code(out.dtype),
                                       _ptr(lse), _stream(stream)), "rf_attn_decode_noalloc")


def rf_row_softmax(x, y, level, work=None, stream=None):
    """x, y [R, n] fp32; work [2R] fp32 for RF_FUSE_NONE."""
    R, n = x.shape
    _need(x, torch.float32, "x")
    _need(y, torch.float32, "y", (R, n))
    if work is not None:
        _need(work, torch.float32, "work", (2 * R,))
    _check(_lib.rf_row_softmax(_ptr(x), R, n, _ptr(y), int(level), _ptr(work), _stream(stream)),
           "rf_row_softmax")


def rf_row_variance(x, mean, var, level, stream=None):
    """x [R, n] fp32 -> mean [R], var [R] (population variance)."""
    R, n = x.shape
    _need(x, torch.float32, "x")
    _need(mean, torch.float32, "mean", (R,))
    _need(var, torch.float32, "var", (R,))
    _check(_lib.rf_row_variance(_ptr(x), R, n, _ptr(mean), _ptr(var), int(level),
                                _stream(stream)), "rf_row_variance")


def rf_moment_of_inertia(mass, pos, center, inertia, level, stream=None):
    """mass [R, n], pos [R, 3, n] fp32 -> center [R, 3], inertia [R]."""
    R, n = mass.shape
    _need(mass, torch.float32, "mass")
    _need(pos, torch.float32, "pos", (R, 3, n))
    _need(center, torch.float32, "center", (R, 3))
    _need(inertia, torch.float32, "inertia", (R,))
    _check(_lib.rf_moment_of_inertia(_ptr(mass), _ptr(pos), R, n, _ptr(center), _ptr(inertia),
                                     int(level), _stream(stream)), "rf_moment_of_inertia")


def rf_layer_norm(x, gamma, beta, eps, y, level, work=None, stream=None):
    """x, y [R, n] fp32; gamma, beta [n]; work [2R] fp32 for RF_FUSE_NONE."""
    R, n = x.shape
    _need(x, torch.float32, "x")
    _need(gamma, torch.float32, "gamma", (n,))
    _need(beta, torch.float32, "beta", (n,))
    _need(y, torch.float32, "y", (R, n))
    if work is not None:
        _need(work, torch.float32, "work", (2 * R,))
    _check(_lib.rf_layer_norm(_ptr(x), _ptr(gamma), _ptr(beta), R, n, float(eps), _ptr(y),
                              int(level), _ptr(work), _stream(stream)), "rf_layer_norm")


def rf_rms_norm(x, gamma, eps, y, level, work=None, stream=None):
    """x, y [R, n] fp32; gamma [n]; level RF_FUSE_NONE needs work [R] fp32."""
    R, n = x.shape
    _need(x, torch.float32, "x")
    _need(gamma, torch.float32, "gamma", (n,))
    _need(y, torch.float32, "y", (R, n))
    if work is not None:
        _need(work, torch.float32, "work", (R,))
    _check(_lib.rf_rms_norm(_ptr(x), _ptr(gamma), R, n, float(eps), _ptr(y), int(level), _ptr(work),
                            _stream(stream)), "rf_rms_norm")


def rf_incremental_quant_fp8_gemm(x, wq, sw, y, sx_final=None, stream=None):
    """x [M, K] bf16, wq [N, K] uint8 e4m3, sw [N] -> y [M, N] bf16, sx_final [M] (optional)."""
    M, K = x.shape
    N = wq.shape[0]
    _need(x, torch.bfloat16, "x")
    _need(wq, torch.uint8, "wq", (N, K))
    _need(sw, torch.float32, "sw", (N,))
    _need(y, torch.bfloat16, "y", (M, N))
    if sx_final is not None:
        _need(sx_final, torch.float32, "sx_final", (M,))
    _check(_lib.rf_incremental_quant_fp8_gemm(_ptr(x), M, K, _ptr(wq), _ptr(sw), N, _ptr(y),
                                              _ptr(sx_final), _stream(stream)),
           "rf_incremental_quant_fp8_gemm")


def rf_decode_segments(groups, keys):
    """A number of segments that fills the current device: ``groups`` =
    B * Hkv * ceil(G / 16) rows of CTAs over up to ``keys`` visible keys each."""
    return _lib.rf_decode_segments(*_c_ints(int(groups), int(keys)))


def _need_cache(q, k, v, lens):
    """Checks q [B, H, D], k/v [B, Hkv, cap, D] and lens [B]; returns the sizes and the device."""
    if q.dim() != 3 or k.dim() != 4:
        raise ValueError("q must be [B, H, D] and k [B, Hkv, cap, D]")
    dev = _device_of(q, "q")
    B, H, D = q.shape
    _, Hkv, cap, _ = k.shape
    dt = q.dtype
    _on(dev, q, dt, q.shape, "q")
    _on(dev, k, dt, (B, Hkv, cap, D), "k")
    _on(dev, v, dt, k.shape, "v")
    if lens is not None:
        _on(dev, lens, torch.int32, (B,), "lens")
    return B, H, Hkv, cap, D, dev


def _need_scratch(dev, B, H, Hkv, D, S, seg_m, seg_l, seg_acc, counters):
    _on(dev, seg_m, torch.float32, (B * H, S), "seg_m")
    _on(dev, seg_l, torch.float32, (B * H, S), "seg_l")
    _on(dev, seg_acc, torch.float32, (B * H, S, D), "seg_acc")
    _on(dev, counters, torch.int32, counters.shape, "counters")
    if counters.numel() < B * Hkv * (-(-(H // max(Hkv, 1)) // 16)):
        raise ValueError("counters must hold B * Hkv * ceil(H / Hkv / 16) elements")


def rf_attn_decode_window(q, k, v, lens, window, sinks, S, scale, seg_m, seg_l, seg_acc, counters,
                          out, lse=None, stream=None):
    """q [B, H, D], k/v [B, Hkv, cap, D] (bf16 or fp16, D = 128), lens int32 [B] or None ->
    out [B, H, D] (q's type or fp32), lse [B, H].  Scratch: seg_m/seg_l [B*H, S],
    seg_acc [B*H, S, D] fp32, counters int32 [B * Hkv * ceil(H / Hkv / 16)], zero at first."""
    B, H, Hkv, cap, D, dev = _need_cache(q, k, v, lens)
    _need_scratch(dev, B, H, Hkv, D, S, seg_m, seg_l, seg_acc, counters)
    _on(dev, out, out.dtype, (B, H, D), "out")
    if lse is not None:
        _on(dev, lse, torch.float32, (B, H), "lse")
    _call_on(dev, stream, "rf_attn_decode_window", _lib.rf_attn_decode_window, q.data_ptr(),
             k.data_ptr(), v.data_ptr(), _addr(lens), *_c_ints(B, H, Hkv, cap, D, window, sinks, S), scale,
             _cache_dtype(q.dtype, "q"), seg_m.data_ptr(), seg_l.data_ptr(), seg_acc.data_ptr(),
             counters.data_ptr(), out.data_ptr(), _cache_dtype(out.dtype, "out"), _addr(lse))


def rf_attn_decode_weights(q, k, v, lens, S, scale, seg_m, seg_l, seg_acc, counters, scores, out,
                           lse, weight, weight_out, stream=None):
    """Decode as rf_attn_decode_window without a window; weight_out [B, Hkv, cap] = weight (or 0
    for None; may be weight_out itself) + the softmax weights summed over each group's heads.
    scores [B, H, cap] fp32 scratch."""
    B, H, Hkv, cap, D, dev = _need_cache(q, k, v, lens)
    _need_scratch(dev, B, H, Hkv, D, S, seg_m, seg_l, seg_acc, counters)
    _on(dev, out, out.dtype, (B, H, D), "out")
    if lse is not None:
        _on(dev, lse, torch.float32, (B, H), "lse")
    _on(dev, scores, torch.float32, (B, H, cap), "scores")
    _on(dev, weight_out, torch.float32, (B, Hkv, cap), "weight_out")
    if weight is not None:
        _on(dev, weight, torch.float32, (B, Hkv, cap), "weight")
    _call_on(dev, stream, "rf_attn_decode_weights", _lib.rf_attn_decode_weights, q.data_ptr(),
             k.data_ptr(), v.data_ptr(), _addr(lens), *_c_ints(B, H, Hkv, cap, D, S), scale,
             _cache_dtype(q.dtype, "q"), seg_m.data_ptr(), seg_l.data_ptr(), seg_acc.data_ptr(),
             counters.data_ptr(), scores.data_ptr(), out.data_ptr(),
             _cache_dtype(out.dtype, "out"), _addr(lse), _addr(weight), weight_out.data_ptr())


def rf_attn_prefill_window(q, k, v, window, sinks, scale, out, lse=None, stream=None):
    """q/out [B, H, N, D], the last N of L positions; k/v [B, Hkv, L, D] (bf16 or fp16, D = 128);
    lse [B, H, N] fp32 (optional)."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, H, N, D] and k [B, Hkv, L, D]")
    dev = _device_of(q, "q")
    B, H, N, D = q.shape
    _, Hkv, L, _ = k.shape
    dt = q.dtype
    _on(dev, q, dt, q.shape, "q")
    _on(dev, k, dt, (B, Hkv, L, D), "k")
    _on(dev, v, dt, k.shape, "v")
    _on(dev, out, dt, q.shape, "out")
    if lse is not None:
        _on(dev, lse, torch.float32, (B, H, N), "lse")
    _call_on(dev, stream, "rf_attn_prefill_window", _lib.rf_attn_prefill_window, q.data_ptr(),
             k.data_ptr(), v.data_ptr(), *_c_ints(B, H, Hkv, N, L, D, window, sinks), scale,
             _cache_dtype(dt, "q"), out.data_ptr(), _addr(lse))


def rf_prefix_segments(B, H, Hkv, prefix):
    """Pieces that rf_attn_decode_shared makes of the prefix on the current device (0: none)."""
    return _lib.rf_prefix_segments(*_c_ints(int(B), int(H), int(Hkv), int(prefix)))


def rf_attn_decode_shared(q, kp, vp, k, v, lens, Sp, S, scale, seg_m, seg_l, seg_acc, counters,
                          out, lse=None, stream=None):
    """q [B, H, D]; kp/vp [Hkv, prefix, D] shared by the batch; k/v [B, Hkv, cap, D] with lens [B]
    own keys -> out [B, H, D], lse [B, H].  Scratch as rf_attn_decode_window with Sp + S pieces."""
    B, H, Hkv, cap, D, dev = _need_cache(q, k, v, lens)
    if kp.dim() != 3:
        raise ValueError("kp must be [Hkv, prefix, D]")
    prefix = kp.shape[1]
    _on(dev, kp, q.dtype, (Hkv, prefix, D), "kp")
    _on(dev, vp, q.dtype, kp.shape, "vp")
    _need_scratch(dev, B, H, Hkv, D, Sp + S, seg_m, seg_l, seg_acc, counters)
    _on(dev, out, out.dtype, (B, H, D), "out")
    if lse is not None:
        _on(dev, lse, torch.float32, (B, H), "lse")
    _call_on(dev, stream, "rf_attn_decode_shared", _lib.rf_attn_decode_shared, q.data_ptr(),
             kp.data_ptr(), vp.data_ptr(), _i32(prefix), k.data_ptr(), v.data_ptr(), _addr(lens),
             *_c_ints(B, H, Hkv, cap, D, Sp, S), scale, _cache_dtype(q.dtype, "q"), seg_m.data_ptr(),
             seg_l.data_ptr(), seg_acc.data_ptr(), counters.data_ptr(), out.data_ptr(),
             _cache_dtype(out.dtype, "out"), _addr(lse))


def _need_evict(dev, k, v, weight, lens, k_out, v_out, weight_out):
    if k.dim() != 4 or k_out.dim() != 4:
        raise ValueError("k and k_out must be [B, Hkv, rows, D]")
    B, Hkv, cap, D = k.shape
    cap_out = k_out.shape[2]
    dt = k.dtype
    _on(dev, k, dt, k.shape, "k")
    _on(dev, k_out, dt, (B, Hkv, cap_out, D), "k_out")
    if v is not None:
        _on(dev, v, dt, k.shape, "v")
    if v_out is not None:
        _on(dev, v_out, dt, k_out.shape, "v_out")
    _on(dev, weight, torch.float32, (B, Hkv, cap), "weight")
    _on(dev, weight_out, torch.float32, (B, Hkv, cap_out), "weight_out")
    if lens is not None:
        _on(dev, lens, torch.int32, (B,), "lens")


def rf_cache_evict(k, v, weight, lens, keep, sinks, recent, k_out, v_out, weight_out, lens_out,
                   kept, stream=None):
    """k/v [B, Hkv, cap, D] (fp32, bf16 or fp16; v None for a cache of one tensor), weight
    [B, Hkv, cap] fp32, lens int32 [B] or None -> k_out/v_out [B, Hkv, cap_out, D], weight_out
    [B, Hkv, cap_out], lens_out int32 [B], kept int32 [B, Hkv, keep]."""
    dev = _device_of(k, "k")
    _need_evict(dev, k, v, weight, lens, k_out, v_out, weight_out)
    B, Hkv, cap, D = k.shape
    _on(dev, lens_out, torch.int32, (B,), "lens_out")
    _on(dev, kept, torch.int32, (B, Hkv, keep), "kept")
    _call_on(dev, stream, "rf_cache_evict", _lib.rf_cache_evict, k.data_ptr(), _addr(v),
             weight.data_ptr(), _addr(lens), *_c_ints(B, Hkv, cap, D), _cache_dtype(k.dtype, "k"),
             *_c_ints(keep, sinks, recent, k_out.shape[2]), k_out.data_ptr(), _addr(v_out), weight_out.data_ptr(),
             lens_out.data_ptr(), kept.data_ptr())


def rf_stream_read(x, out_xor, stream=None):
    """XOR every 32-bit word of the CUDA tensor ``x`` into ``out_xor`` (one
    int32 element, device memory) with one streaming read of ``x``."""
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor")
    _need(out_xor, torch.int32, "out_xor", (1,))
    _check(_lib.rf_stream_read(_ptr(x), x.numel() * x.element_size(), _ptr(out_xor),
                               _stream(stream)), "rf_stream_read")


def rf_selftest_wait_timeout(waited_ms, stream=None):
    """waited_ms: int32 CUDA tensor of one element; the timeout shows up in rf_device_error()."""
    _need(waited_ms, torch.int32, "waited_ms", (1,))
    _check(_lib.rf_selftest_wait_timeout(_ptr(waited_ms), _stream(stream)), "rf_selftest_wait_timeout")


def rf_selftest_bounds(stream=None):
    """One refused index through the bounds check (bounds-checked build only);
    RF_ERR_BOUNDS then shows up in rf_device_error()."""
    _check(_lib.rf_selftest_bounds(_stream(stream)), "rf_selftest_bounds")


def rf_bounds_checked():
    """True if the loaded library checks every kernel's global indices."""
    return bool(_lib.rf_bounds_checked())


def rf_device_error(stream=None):
    """Synchronise and return (and clear) the on-device status words: bounded
    waits, and in the bounds-checked build the index checks."""
    st = _I(0)
    _check(_lib.rf_device_error(ctypes.byref(st), _stream(stream)), "rf_device_error")
    return st.value


# ----------------------------------------------------- convenience wrappers --

def attn_decode(q, k, v, S, scale, out_dtype=None, return_states=False, stream=None):
    """Split-KV decode: rf_attn_decode_split then rf_state_merge.

    q [R, D], k/v [R, L, D]; returns out [R, D] (and lse, and the segment states
    if ``return_states``)."""
    R, L, D = k.shape
    dev = k.device
    seg_m = torch.empty(R, S, device=dev, dtype=torch.float32)
    seg_l = torch.empty(R, S, device=dev, dtype=torch.float32)
    seg_acc = torch.empty(R, S, D, device=dev, dtype=torch.float32)
    out = torch.empty(R, D, device=dev, dtype=out_dtype or k.dtype)
    lse = torch.empty(R, device=dev, dtype=torch.float32)
    rf_attn_decode_split(q, k, v, S, scale, seg_m, seg_l, seg_acc, stream)
    rf_state_merge(seg_m, seg_l, seg_acc, out, lse, stream)
    if return_states:
        return out, lse, (seg_m, seg_l, seg_acc)
    return out, lse


def mla_decode(q, c, S, scale, dv=512, return_states=False, stream=None):
    """MLA split decode: rf_mla_decode_split then rf_state_merge.

    q [B, H, 576], c [B, L, 576] bf16; returns out [B, H, dv] bf16 and lse [B, H]
    (and the segment states if ``return_states``)."""
    B, H, _ = q.shape
    dev = q.device
    seg_m = torch.empty(B, H, S, device=dev, dtype=torch.float32)
    seg_l = torch.empty(B, H, S, device=dev, dtype=torch.float32)
    seg_acc = torch.empty(B, H, S, dv, device=dev, dtype=torch.float32)
    out = torch.empty(B, H, dv, device=dev, dtype=torch.bfloat16)
    lse = torch.empty(B, H, device=dev, dtype=torch.float32)
    rf_mla_decode_split(q, c, S, scale, seg_m, seg_l, seg_acc, stream)
    rf_state_merge(seg_m.view(B * H, S), seg_l.view(B * H, S), seg_acc.view(B * H, S, dv),
                   out.view(B * H, dv), lse.view(B * H), stream)
    if return_states:
        return out, lse, (seg_m, seg_l, seg_acc)
    return out, lse


def softmax_topk(logits, k, renormalize=True, stream=None):
    T = logits.shape[0]
    idx = torch.empty(T, k, device=logits.device, dtype=torch.int32)
    w = torch.empty(T, k, device=logits.device, dtype=torch.float32)
    rf_softmax_topk(logits, k, renormalize, idx, w, stream)
    return idx, w


def absmax_quant_fp8_gemm(x, wq, sw, stream=None):
    M, K = x.shape
    N = wq.shape[0]
    xq = torch.empty(M, K, device=x.device, dtype=torch.uint8)
    sx = torch.empty(M, device=x.device, dtype=torch.float32)
    y = torch.empty(M, N, device=x.device, dtype=torch.bfloat16)
    rf_absmax_quant_fp8_gemm(x, wq, sw, xq, sx, y, stream)
    return xq, sx, y


def attn_prefill(q, k, v, causal=True, scale=None, stream=None):
    B, H, N, D = q.shape
    if scale is None:
        scale = D ** -0.5
    out = torch.empty_like(q)
    lse = torch.empty(B, H, N, device=q.device, dtype=torch.float32)
    rf_attn_prefill(q, k, v, causal, scale, out, lse, stream)
    return out, lse


class DecodeWorkspace(typing.NamedTuple):
    """Scratch of one decode call over a cache of grouped heads (decode_workspace makes it):
    states of up to ``prefix_S`` + ``S`` pieces per row, zeroed counters and, where asked for, a
    score per head and key.  A serving loop keeps one per call that may be in flight at a time."""
    S: int
    prefix_S: int
    seg_m: torch.Tensor
    seg_l: torch.Tensor
    seg_acc: torch.Tensor
    counters: torch.Tensor
    scores: torch.Tensor
    sizes: tuple        # (device index, B, H, Hkv, D)
    addresses: tuple    # of seg_m, seg_l, seg_acc, counters

    def check(self, *sizes):
        if sizes != self.sizes:
            raise ValueError(f"work was made for (device, B, H, Hkv, D) = {self.sizes}, "
                             f"the call has {sizes}")


def decode_workspace(B, H, Hkv, cap, D=128, prefix=0, window=0, sinks=0, weights=False, S=None,
                     device=None):
    """Scratch for attn_decode_window (window, sinks as in the call), attn_decode_shared (the
    prefix's length) or attn_decode_weights (weights=True).  S pieces per row (None: as many as
    fill the device).  The counters are zeroed on the current stream: a call on another stream
    has to come after that."""
    if H < 1 or Hkv < 1 or H % Hkv:
        raise ValueError("H must be a positive multiple of Hkv")
    with torch.cuda.device(torch.device("cuda" if device is None else device)):
        dev = torch.device("cuda", torch.cuda.current_device())
        if S is None:
            keys = min(cap, window + sinks) if window else cap
            S = rf_decode_segments(B * Hkv * (-(-(H // Hkv) // 16)), keys)
        prefix_S = rf_prefix_segments(B, H, Hkv, prefix) if prefix else 0
        f32 = dict(device=dev, dtype=torch.float32)
        seg_m, seg_l = (torch.empty(B * H, prefix_S + S, **f32) for _ in range(2))
        seg_acc = torch.empty(B * H, prefix_S + S, D, **f32)
        counters = torch.zeros(B * Hkv * (-(-(H // Hkv) // 16)), device=dev, dtype=torch.int32)
        scores = torch.empty(B, H, cap, **f32) if weights else None
        return DecodeWorkspace(S, prefix_S, seg_m, seg_l, seg_acc, counters, scores,
                               (dev.index, B, H, Hkv, D),
                               tuple(t.data_ptr() for t in (seg_m, seg_l, seg_acc, counters)))


def _within(stream, t, call, *args, **kwargs):
    """call(*args, **kwargs) with ``stream`` current, so that what it allocates belongs to that
    stream and is not handed out again while the stream still uses it."""
    if stream.device != t.device:
        raise ValueError(f"stream of {stream.device} for tensors on {t.device}")
    with torch.cuda.stream(stream):
        return call(*args, **kwargs)


def _done(r, where):
    """The outputs of a quick call, whose result is a status where it was refused."""
    if type(r) is not tuple:
        raise RFError(r, where)
    return r


def _outputs(q, out_dtype):
    out = torch.empty_like(q) if out_dtype is None else torch.empty_like(q, dtype=out_dtype)
    return out, torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)


def attn_decode_window(q, k, v, lens=None, window=0, sinks=0, scale=None, work=None,
                       out_dtype=None, stream=None):
    """Single-token decode over the visible keys of a ragged batch of caches.

    q [B, H, D], k/v [B, Hkv, cap, D] (bf16 or fp16), lens int32 [B] (None: all cap rows in use).
    Key j is visible if it is one of the last ``window`` (0: all) or of the first ``sinks``.
    Returns out [B, H, D] and lse [B, H]; ``work`` from decode_workspace saves its allocation."""
    if stream is not None:
        return _within(stream, q, attn_decode_window, q, k, v, lens, window, sinks, scale, work,
                       out_dtype)
    if _calls is not None and work is not None and out_dtype is None:
        r = _calls.decode_window(_DECODE_WINDOW, q, k, v, lens, window, sinks, scale, work.S, work.sizes,
                                 work.addresses)
        if r is not None:
            return _done(r, "rf_attn_decode_window")
    B, H, Hkv, cap, D, dev = _need_cache(q, k, v, lens)
    if work is None:
        work = decode_workspace(B, H, Hkv, cap, D, window=window, sinks=sinks, device=q.device)
    work.check(dev, B, H, Hkv, D)
    out, lse = _outputs(q, out_dtype)
    _call_on(dev, None, "rf_attn_decode_window", _lib.rf_attn_decode_window, q.data_ptr(),
             k.data_ptr(), v.data_ptr(), _addr(lens), *_c_ints(B, H, Hkv, cap, D, window, sinks, work.S),
             D ** -0.5 if scale is None else scale, _cache_dtype(q.dtype, "q"), *work.addresses,
             out.data_ptr(), _cache_dtype(out.dtype, "out"), lse.data_ptr())
    return out, lse


def attn_prefill_window(q, k, v, window=0, sinks=0, scale=None, stream=None):
    """Attention of the last N of L positions over their visible keys: one of the ``window`` keys
    up to the position itself (0: all) or one of the first ``sinks``.

    q [B, H, N, D], k/v [B, Hkv, L, D] (bf16 or fp16).  Returns out [B, H, N, D] and lse [B, H, N]."""
    if stream is not None:
        return _within(stream, q, attn_prefill_window, q, k, v, window, sinks, scale)
    if _calls is not None:
        r = _calls.prefill_window(_PREFILL_WINDOW, q, k, v, window, sinks, scale)
        if r is not None:
            return _done(r, "rf_attn_prefill_window")
    out, lse = _outputs(q, None)
    rf_attn_prefill_window(q, k, v, window, sinks, q.shape[-1] ** -0.5 if scale is None else scale,
                           out, lse)
    return out, lse


def attn_decode_shared(q, kp, vp, k, v, lens=None, scale=None, work=None, out_dtype=None,
                       stream=None):
    """Single-token decode for a batch whose sequences share their first keys.

    q [B, H, D]; kp/vp [Hkv, prefix, D]; k/v [B, Hkv, cap, D] with lens [B] own keys behind the
    prefix (None: cap; 0 allowed).  Returns out [B, H, D] and lse [B, H]."""
    if stream is not None:
        return _within(stream, q, attn_decode_shared, q, kp, vp, k, v, lens, scale, work, out_dtype)
    if _calls is not None and work is not None and out_dtype is None:
        r = _calls.decode_shared(_DECODE_SHARED, q, kp, vp, k, v, lens, scale, work.prefix_S, work.S,
                                 work.sizes, work.addresses)
        if r is not None:
            return _done(r, "rf_attn_decode_shared")
    B, H, Hkv, cap, D, dev = _need_cache(q, k, v, lens)
    if kp.dim() != 3:
        raise ValueError("kp must be [Hkv, prefix, D]")
    prefix = kp.shape[1]
    _on(dev, kp, q.dtype, (Hkv, prefix, D), "kp")
    _on(dev, vp, q.dtype, kp.shape, "vp")
    if work is None:
        work = decode_workspace(B, H, Hkv, cap, D, prefix=prefix, device=q.device)
    work.check(dev, B, H, Hkv, D)
    out, lse = _outputs(q, out_dtype)
    _call_on(dev, None, "rf_attn_decode_shared", _lib.rf_attn_decode_shared, q.data_ptr(),
             kp.data_ptr(), vp.data_ptr(), _i32(prefix), k.data_ptr(), v.data_ptr(), _addr(lens),
             *_c_ints(B, H, Hkv, cap, D, work.prefix_S, work.S), D ** -0.5 if scale is None else scale,
             _cache_dtype(q.dtype, "q"), *work.addresses, out.data_ptr(),
             _cache_dtype(out.dtype, "out"), lse.data_ptr())
    return out, lse


def attn_decode_weights(q, k, v, lens=None, weight=None, scale=None, work=None, weight_out=None,
                        out_dtype=None, stream=None):
    """Single-token decode that also totals each key's attention weight.

    Returns out [B, H, D], lse [B, H] and weight_out [B, Hkv, cap] = weight (None: 0) plus the
    softmax weights of this token, summed over each key head's query heads; ``weight_out`` may be
    ``weight`` itself."""
    if stream is not None:
        return _within(stream, q, attn_decode_weights, q, k, v, lens, weight, scale, work, weight_out,
                       out_dtype)
    if _calls is not None and work is not None and out_dtype is None and weight_out is None:
        r = _calls.decode_weights(_DECODE_WEIGHTS, q, k, v, lens, weight, scale, work.S, work.sizes,
                                  work.addresses, work.scores)
        if r is not None:
            return _done(r, "rf_attn_decode_weights")
    B, H, Hkv, cap, D, dev = _need_cache(q, k, v, lens)
    if weight is not None:
        _on(dev, weight, torch.float32, (B, Hkv, cap), "weight")
    if work is None:
        work = decode_workspace(B, H, Hkv, cap, D, weights=True, device=q.device)
    work.check(dev, B, H, Hkv, D)
    if work.scores is None or work.scores.shape[2] != cap:
        raise ValueError("work must come from decode_workspace(..., cap, weights=True)")
    out, lse = _outputs(q, out_dtype)
    if weight_out is None:
        weight_out = torch.empty((B, Hkv, cap), device=q.device, dtype=torch.float32)
    else:
        _on(dev, weight_out, torch.float32, (B, Hkv, cap), "weight_out")
    _call_on(dev, None, "rf_attn_decode_weights", _lib.rf_attn_decode_weights, q.data_ptr(),
             k.data_ptr(), v.data_ptr(), _addr(lens), *_c_ints(B, H, Hkv, cap, D, work.S),
             D ** -0.5 if scale is None else scale, _cache_dtype(q.dtype, "q"), *work.addresses,
             work.scores.data_ptr(), out.data_ptr(), _cache_dtype(out.dtype, "out"),
             lse.data_ptr(), _addr(weight), weight_out.data_ptr())
    return out, lse, weight_out


def cache_evict(k, v, weight, lens, keep, sinks=0, recent=0, cap_out=None, out=None, stream=None):
    """Keep ``keep`` rows per sequence and key head: the first ``sinks``, the last ``recent`` and
    the rows of largest weight between them, in their old order.

    k/v [B, Hkv, cap, D] (v may be None), weight [B, Hkv, cap], lens int32 [B] or None.  Returns
    k_out, v_out, weight_out (``out`` if given, else new zeroed tensors of cap_out = keep rows by
    default), lens_out [B] and kept [B, Hkv, keep] (source rows, -1 behind a short sequence)."""
    if stream is not None:
        return _within(stream, k, cache_evict, k, v, weight, lens, keep, sinks, recent, cap_out, out)
    if _calls is not None and out is not None:
        r = _calls.cache_evict(_CACHE_EVICT, k, v, weight, lens, keep, sinks, recent, *out)
        if r is not None:
            return (*out, *_done(r, "rf_cache_evict"))
    if k.dim() != 4:
        raise ValueError("k must be [B, Hkv, rows, D]")
    dev = _device_of(k, "k")
    B, Hkv, cap, D = k.shape
    if out is None:
        rows = keep if cap_out is None else cap_out
        new = dict(device=k.device, dtype=k.dtype)
        out = (torch.zeros(B, Hkv, rows, D, **new),
               None if v is None else torch.zeros(B, Hkv, rows, D, **new),
               torch.zeros(B, Hkv, rows, device=k.device))
    k_out, v_out, weight_out = out
    _need_evict(dev, k, v, weight, lens, k_out, v_out, weight_out)
    new = dict(device=k.device, dtype=torch.int32)
    lens_out, kept = torch.empty(B, **new), torch.empty((B, Hkv, keep), **new)
    _call_on(dev, None, "rf_cache_evict", _lib.rf_cache_evict, k.data_ptr(), _addr(v),
             weight.data_ptr(), _addr(lens), *_c_ints(B, Hkv, cap, D), _cache_dtype(k.dtype, "k"),
             *_c_ints(keep, sinks, recent, k_out.shape[2]), k_out.data_ptr(), _addr(v_out), weight_out.data_ptr(),
             lens_out.data_ptr(), kept.data_ptr())
    return k_out, v_out, weight_out, lens_out, kept
