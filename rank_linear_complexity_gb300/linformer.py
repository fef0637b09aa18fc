"""Python binding of the C ABI in include/linformer_attn.h (argument marshalling only).

Every function here converts its arguments to pointers and integers and calls
the CUDA library of the same name; all computation runs in the library's
kernels.  Importing this module does not load the library; the first call does,
and raises if the library has not been built (there is no other implementation
to fall back to).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

PER_HEAD, KV, HEADWISE, LAYERWISE = 0, 1, 2, 3
F32, BF16, BF16_F32OUT = 0, 1, 2
PATH_SIMT, PATH_TENSOR = 0, 1
KERNEL_COUNT = 12
ROTARY_HALVES, ROTARY_INTERLEAVED = 0, 1
ROTARY_PLAIN, ROTARY_LINEAR, ROTARY_BASE, ROTARY_BY_PARTS = 0, 1, 2, 3

_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_d = ctypes.c_double

SYMBOLS = [
    "linformer_attn_fwd", "linformer_project_fwd", "linformer_attn_fwd_host",
    "linformer_select_path", "linformer_status_string", "linformer_debug_read_device_status",
    "linformer_set_pv_terms", "linformer_launch_count", "linformer_profile_enable",
    "linformer_profile_collect", "linformer_kernel_name", "linformer_attn_fwd_noalloc",
    "linformer_window_projection", "linformer_attn_bwd", "linformer_dense_attn_fwd",
    "linformer_pool_peak_bytes", "linformer_debug_wait_probe", "linformer_softmax_attn_fwd",
    "linformer_softmax_attn_bwd", "linformer_rotary", "linformer_rotary_phase",
    "linformer_cache_append", "linformer_cache_keep", "linformer_paged_attn_fwd",
    "linformer_tree_attn_fwd", "linformer_tree_mask", "linformer_cache_packed",
]


class LinformerError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it was never built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(
                    f"CUDA library not built ({path} missing): run "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(path)
            fwd_args = [_vp] * 5 + [_vp, _vp] + [_i] * 7 + [_vp]
            L.linformer_attn_fwd.argtypes = fwd_args
            L.linformer_attn_fwd.restype = _i
            L.linformer_attn_fwd_host.argtypes = fwd_args
            L.linformer_attn_fwd_host.restype = _i
            L.linformer_attn_fwd_noalloc.argtypes = fwd_args
            L.linformer_attn_fwd_noalloc.restype = _i
            L.linformer_project_fwd.argtypes = [_vp] * 5 + [_vp, _vp] + [_i] * 7 + [_vp]
            L.linformer_project_fwd.restype = _i
            L.linformer_select_path.argtypes = [_i] * 7
            L.linformer_select_path.restype = _i
            L.linformer_status_string.argtypes = [_i]
            L.linformer_status_string.restype = ctypes.c_char_p
            L.linformer_debug_read_device_status.argtypes = [_vp]
            L.linformer_debug_read_device_status.restype = _i
            L.linformer_set_pv_terms.argtypes = [_i]
            L.linformer_set_pv_terms.restype = _i
            L.linformer_launch_count.argtypes = []
            L.linformer_launch_count.restype = ctypes.c_int64
            L.linformer_profile_enable.argtypes = [_i]
            L.linformer_profile_enable.restype = _i
            L.linformer_profile_collect.argtypes = [ctypes.POINTER(ctypes.c_double),
                                                    ctypes.POINTER(ctypes.c_int64)]
            L.linformer_profile_collect.restype = _i
            L.linformer_dense_attn_fwd.argtypes = [_vp] * 5 + [_i] * 5 + [_vp]
            L.linformer_dense_attn_fwd.restype = _i
            L.linformer_debug_wait_probe.argtypes = [_vp]
            L.linformer_debug_wait_probe.restype = _i
            L.linformer_pool_peak_bytes.argtypes = [_i]
            L.linformer_pool_peak_bytes.restype = ctypes.c_int64
            L.linformer_attn_bwd.argtypes = [_vp] * 12 + [_i] * 7 + [_vp]
            L.linformer_attn_bwd.restype = _i
            L.linformer_window_projection.argtypes = [_vp, _vp, _i, _i, _i, _vp]
            L.linformer_window_projection.restype = _i
            L.linformer_softmax_attn_fwd.argtypes = ([_vp] * 11 + [_i] * 6 + [_f] + [_i] * 3
                                                     + [_vp])
            L.linformer_softmax_attn_fwd.restype = _i
            L.linformer_softmax_attn_bwd.argtypes = ([_vp] * 19 + [_i] * 6 + [_f] + [_i] * 3
                                                     + [_vp])
            L.linformer_softmax_attn_bwd.restype = _i
            L.linformer_rotary.argtypes = ([_vp] * 4 + [_i] + [_vp] * 4 + [_i] + [_vp] * 2
                                           + [_i] * 6 + [_f] + [_i] * 2 + [_vp])
            L.linformer_rotary.restype = _i
            L.linformer_rotary_phase.argtypes = [_vp, _i, _d, _i, _d, _i, _d, _d, _vp]
            L.linformer_rotary_phase.restype = _i
            L.linformer_cache_append.argtypes = [_vp] * 17 + [_i] * 10 + [_f, _i, _vp]
            L.linformer_cache_append.restype = _i
            L.linformer_cache_keep.argtypes = [_vp] * 8 + [_i] * 8 + [_vp]
            L.linformer_cache_keep.restype = _i
            L.linformer_paged_attn_fwd.argtypes = [_vp] * 12 + [_i] * 8 + [_f] + [_i] * 3 + [_vp]
            L.linformer_paged_attn_fwd.restype = _i
            L.linformer_tree_attn_fwd.argtypes = [_vp] * 13 + [_i] * 8 + [_f, _i, _vp]
            L.linformer_tree_attn_fwd.restype = _i
            L.linformer_tree_mask.argtypes = [_vp] * 2 + [_i] * 2 + [_vp]
            L.linformer_tree_mask.restype = _i
            L.linformer_cache_packed.argtypes = [_i, ctypes.c_char_p, _i]
            L.linformer_cache_packed.restype = _i
            L.linformer_kernel_name.argtypes = [_i]
            L.linformer_kernel_name.restype = ctypes.c_char_p
            _lib = L
    return _lib


def _ptr(x):
    """Device/host address of a tensor (or an int address, or None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def linformer_attn_fwd(Q, K, V, E, F, pad_lengths, O, b, h, n, d, k, share_mode, dtype,
                       stream=None) -> int:
    return lib().linformer_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(E), _ptr(F),
                                    _ptr(pad_lengths), _ptr(O), b, h, n, d, k, share_mode,
                                    dtype, _stream_handle(stream))


def linformer_project_fwd(K, V, E, F, pad_lengths, Kbar, Vbar, b, h, n, d, k, share_mode,
                          dtype, stream=None) -> int:
    return lib().linformer_project_fwd(_ptr(K), _ptr(V), _ptr(E), _ptr(F), _ptr(pad_lengths),
                                       _ptr(Kbar), _ptr(Vbar), b, h, n, d, k, share_mode,
                                       dtype, _stream_handle(stream))


def linformer_attn_fwd_host(Q, K, V, E, F, pad_lengths, O, b, h, n, d, k, share_mode, dtype,
                            stream=None) -> int:
    return lib().linformer_attn_fwd_host(_ptr(Q), _ptr(K), _ptr(V), _ptr(E), _ptr(F),
                                         _ptr(pad_lengths), _ptr(O), b, h, n, d, k,
                                         share_mode, dtype, _stream_handle(stream))


def linformer_attn_fwd_noalloc(Q, K, V, E, F, pad_lengths, O, b, h, n, d, k, share_mode,
                               dtype, stream=None) -> int:
    """Same as linformer_attn_fwd, with the library's fixed device workspace (no allocation)."""
    return lib().linformer_attn_fwd_noalloc(_ptr(Q), _ptr(K), _ptr(V), _ptr(E), _ptr(F),
                                            _ptr(pad_lengths), _ptr(O), b, h, n, d, k,
                                            share_mode, dtype, _stream_handle(stream))


def linformer_select_path(b, h, n, d, k, share_mode, dtype) -> int:
    return lib().linformer_select_path(b, h, n, d, k, share_mode, dtype)


def status_string(status: int) -> str:
    try:
        return lib().linformer_status_string(status).decode()
    except Exception:  # library unavailable: still give a message
        return "unknown"


def linformer_debug_read_device_status(stream=None) -> int:
    return lib().linformer_debug_read_device_status(_stream_handle(stream))


def linformer_debug_wait_probe(stream=None) -> int:
    return lib().linformer_debug_wait_probe(_stream_handle(stream))


def linformer_set_pv_terms(terms: int) -> int:
    return lib().linformer_set_pv_terms(terms)


def linformer_launch_count() -> int:
    return lib().linformer_launch_count()


def linformer_profile_enable(enable: bool) -> int:
    return lib().linformer_profile_enable(1 if enable else 0)


def linformer_profile_collect():
    """Returns {kernel name: (total ms, launches)} for kernels that ran."""
    ms = (ctypes.c_double * KERNEL_COUNT)()
    cnt = (ctypes.c_int64 * KERNEL_COUNT)()
    st = lib().linformer_profile_collect(ms, cnt)
    if st != 0:
        raise LinformerError(st, "linformer_profile_collect")
    out = {}
    for i in range(KERNEL_COUNT):
        if cnt[i]:
            out[lib().linformer_kernel_name(i).decode()] = (ms[i], cnt[i])
    return out


# --- tensor-level conveniences (still marshalling only) ------------------------------

def _dims(Q, E, share_mode):
    b, h, n, d = Q.shape
    k = E.shape[-2]
    return b, h, n, d, k


def dtype_code(t, out_fp32: bool = False) -> int:
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16_F32OUT if out_fp32 else BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def attention(Q, K, V, E, F=None, lengths=None, share_mode: int = PER_HEAD,
              out_fp32: bool = False, out=None, stream=None):
    """O = Linformer attention of device tensors Q, K, V [b][h][n][d] (allocates O)."""
    import torch
    b, h, n, d, k = _dims(Q, E, share_mode)
    code = dtype_code(Q, out_fp32)
    if out is None:
        odt = torch.bfloat16 if code == BF16 else torch.float32
        out = torch.empty((b, h, n, d), dtype=odt, device=Q.device)
    st = linformer_attn_fwd(Q, K, V, E, F, lengths, out, b, h, n, d, k, share_mode, code,
                            stream)
    if st != 0:
        raise LinformerError(st, "linformer_attn_fwd")
    return out


def projection(K, V, E, F=None, lengths=None, share_mode: int = PER_HEAD, stream=None):
    """(Kbar, Vbar) fp32 [b][h][k][d] of device tensors K, V."""
    import torch
    b, h, n, d = K.shape
    k = E.shape[-2]
    Kb = torch.empty((b, h, k, d), dtype=torch.float32, device=K.device)
    Vb = torch.empty_like(Kb)
    st = linformer_project_fwd(K, V, E, F, lengths, Kb, Vb, b, h, n, d, k, share_mode,
                               dtype_code(K), stream)
    if st != 0:
        raise LinformerError(st, "linformer_project_fwd")
    return Kb, Vb


def linformer_window_projection(P, weights, n, k, dtype, stream=None) -> int:
    return lib().linformer_window_projection(_ptr(P), _ptr(weights), n, k, dtype,
                                             _stream_handle(stream))


def window_projection(n: int, k: int, weights=None, dtype=None, device="cuda", stream=None):
    """[k][n] device tensor: mean pooling (weights None) or a convolution with kernel =
    stride = n / k (weights: float32 device tensor of n / k values), to pass as E (and F)."""
    import torch
    dt = torch.bfloat16 if dtype is None else dtype
    P = torch.empty((k, n), dtype=dt, device=device)
    code = F32 if dt == torch.float32 else BF16
    st = linformer_window_projection(P, weights, n, k, code, stream)
    if st != 0:
        raise LinformerError(st, "linformer_window_projection")
    return P


def linformer_attn_bwd(Q, K, V, E, F, pad_lengths, dO, dQ, dK, dV, dE, dF, b, h, n, d, k,
                       share_mode, dtype, stream=None) -> int:
    return lib().linformer_attn_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(E), _ptr(F),
                                    _ptr(pad_lengths), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV),
                                    _ptr(dE), _ptr(dF), b, h, n, d, k, share_mode, dtype,
                                    _stream_handle(stream))


def attention_backward(Q, K, V, E, F, lengths, dO, share_mode: int = PER_HEAD, stream=None):
    """(dQ, dK, dV, dE, dF) of device fp32 tensors; dF is None when F is E (KV, LAYERWISE)."""
    import torch
    b, h, n, d, k = _dims(Q, E, share_mode)
    dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    dE = torch.empty_like(E)
    distinct = share_mode in (PER_HEAD, HEADWISE)
    dF = torch.empty_like(F if F is not None else E) if distinct else None
    st = linformer_attn_bwd(Q, K, V, E, F, lengths, dO, dQ, dK, dV, dE, dF, b, h, n, d, k,
                            share_mode, dtype_code(Q), stream)
    if st != 0:
        raise LinformerError(st, "linformer_attn_bwd")
    return dQ, dK, dV, dE, dF


def linformer_dense_attn_fwd(Q, K, V, pad_lengths, O, b, h, n, d, dtype, stream=None) -> int:
    return lib().linformer_dense_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(pad_lengths), _ptr(O),
                                          b, h, n, d, dtype, _stream_handle(stream))


def linformer_pool_peak_bytes(reset: bool = False) -> int:
    return lib().linformer_pool_peak_bytes(1 if reset else 0)


def dense_attention(Q, K, V, lengths=None, out=None, stream=None):
    """O = softmax(Q K^T / sqrt(d)) V of device fp32 tensors [b][h][n][d] (allocates O)."""
    import torch
    b, h, n, d = Q.shape
    if out is None:
        out = torch.empty((b, h, n, d), dtype=torch.float32, device=Q.device)
    st = linformer_dense_attn_fwd(Q, K, V, lengths, out, b, h, n, d, dtype_code(Q), stream)
    if st != 0:
        raise LinformerError(st, "linformer_dense_attn_fwd")
    return out


# --- exact softmax attention and rotary positions (strided [b][h][n][d] tensors) ------------
#
# Calls of a few microseconds, so these marshal with care: no closures, strides by value from a
# small table, the current stream from the binding that torch.cuda.current_stream() wraps
# (1 us instead of 6), one comparison of shapes where one says it all.
#
# The calls return once launched.  A wait inside a kernel that ran out (2 s) leaves rows of the
# outputs unwritten and is recorded in the device status word: linformer_debug_read_device_status()
# synchronises, reads and clears it.
#
# A call given a stream (an object or a handle) runs with that stream as the current one: tensors
# that it makes belong to the stream, as those of any torch operation would.  Its inputs have to be
# ready there, and kept until the stream has read them.

_stride_table = {}   # (batch, head, row) strides -> address of an int64[3]
_stride_arrays = []  # which holds them


def _strides(x):
    """Address of the tensor's batch, head and row strides (None: dense)."""
    if x.is_contiguous():
        return None
    key = x.stride()
    at = _stride_table.get(key)
    if at is None:
        if key[3] != 1:
            raise ValueError("the last dimension has to be contiguous")
        arr = (ctypes.c_int64 * 3)(*key[:3])
        if len(_stride_table) >= 4096:
            return arr  # for this call alone: no entry is ever taken out, another call may hold it
        _stride_arrays.append(arr)
        at = _stride_table[key] = ctypes.addressof(arr)
    return at


def _current_on(device, stream):
    """Context that makes `stream` the current one."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"CUDA tensors are needed, got {device}")
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream)
        # (0 and 1 are the default stream's handles, under its own name in torch)
        stream = (torch.cuda.default_stream(device) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device))
    if device.index is not None and stream.device != device:
        raise ValueError(f"a stream of {stream.device} for tensors on {device}")
    return torch.cuda.stream(stream)


def _stream_of(device, *tensors):
    """The current stream's handle, after a check that the tensors (None: not given) are on
    `device`."""
    if device.type != "cuda":
        raise ValueError(f"CUDA tensors are needed, got {device}")
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {device} and {t.device}")
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(index)
    except AttributeError:  # a private name
        return torch.cuda.current_stream(device).cuda_stream


def _call(fn, device, args, name):
    """fn(*args) with `device` current (the library works on the current device)."""
    import torch
    try:
        current = torch._C._cuda_getDevice()
    except AttributeError:  # a private name
        current = torch.cuda.current_device()
    if current == device.index:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st != 0:
        raise LinformerError(st, name)


def _int32(name, x):
    """Refuses what would not survive the passage to a C int."""
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} = {x} is outside the 32-bit range")
    return x


def _sizes(name, shape):
    if max(shape) > 0x7fffffff:
        raise ValueError(f"{name}: a size of {tuple(shape)} is outside the 32-bit range")


def _check(name, x, shape, dtype):
    if x.shape != shape or x.dtype != dtype:
        raise ValueError(f"{name}: {dtype} of shape {tuple(shape)} is needed, got {x.dtype} of "
                         f"{tuple(x.shape)}")


def _check_dense(name, x, shape, dtype):
    _check(name, x, shape, dtype)
    if not x.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is needed")


def softmax_attention(Q, K, V, q_lengths=None, k_lengths=None, causal: bool = False,
                      window: int = 0, scale=None, out=None, lse=None, stream=None):
    """(O, lse) of the exact attention of Q [b][hq][n][d] over K, V [b][hk][m][d] (bf16, any
    strides): O shaped like Q, lse fp32 [b][hq][n] as softmax_attention_backward takes it.

    causal: the valid parts end together (the last query sees every key), with window > 0
    only the last `window` keys up to its own.  scale defaults to 1 / sqrt(d)."""
    import torch
    if stream is not None:
        with _current_on(Q.device, stream):
            return softmax_attention(Q, K, V, q_lengths, k_lengths, causal, window, scale, out, lse)
    shape, kv, dtype, device = Q.shape, K.shape, Q.dtype, Q.device
    b, hq, n, d = shape
    _, hk, m, _ = kv
    _sizes("Q", shape)
    _sizes("K", kv)
    handle = _stream_of(device, K, V, q_lengths, k_lengths, out, lse)
    if kv[0] != b or kv[3] != d or K.dtype != dtype:
        _check("K", K, (b, hk, m, d), dtype)
    _check("V", V, kv, dtype)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    else:
        _check("out", out, shape, dtype)
    if lse is None:
        lse = torch.empty((b, hq, n), dtype=torch.float32, device=device)
    else:
        _check_dense("lse", lse, (b, hq, n), torch.float32)
    if q_lengths is not None:
        _check_dense("q_lengths", q_lengths, (b,), torch.int32)
        q_lengths = q_lengths.data_ptr()
    if k_lengths is not None:
        _check_dense("k_lengths", k_lengths, (b,), torch.int32)
        k_lengths = k_lengths.data_ptr()
    _call(lib().linformer_softmax_attn_fwd, device,
          (Q.data_ptr(), _strides(Q), K.data_ptr(), _strides(K), V.data_ptr(), _strides(V),
           out.data_ptr(), _strides(out), lse.data_ptr(), q_lengths, k_lengths, b, hq, hk, n, m, d,
           d ** -0.5 if scale is None else scale, 1 if causal else 0,
           _int32("window", window), dtype_code(Q), handle),
          "linformer_softmax_attn_fwd")
    return out, lse


def softmax_attention_backward(Q, K, V, O, dO, lse, q_lengths=None, k_lengths=None,
                               causal: bool = False, window: int = 0, scale=None, dQ=None,
                               dK=None, dV=None, stream=None):
    """(dQ, dK, dV) from the inputs and results of softmax_attention and dO = dLoss/dO."""
    import torch
    if stream is not None:
        with _current_on(Q.device, stream):
            return softmax_attention_backward(Q, K, V, O, dO, lse, q_lengths, k_lengths, causal,
                                              window, scale, dQ, dK, dV)
    shape, kv, dtype, device = Q.shape, K.shape, Q.dtype, Q.device
    b, hq, n, d = shape
    _, hk, m, _ = kv
    _sizes("Q", shape)
    _sizes("K", kv)
    handle = _stream_of(device, K, V, O, dO, lse, q_lengths, k_lengths, dQ, dK, dV)
    if kv[0] != b or kv[3] != d or K.dtype != dtype:
        _check("K", K, (b, hk, m, d), dtype)
    _check("V", V, kv, dtype)
    _check("O", O, shape, dtype)
    _check("dO", dO, shape, dtype)
    _check_dense("lse", lse, (b, hq, n), torch.float32)
    if dQ is None:
        dQ = torch.empty(shape, dtype=dtype, device=device)
    else:
        _check("dQ", dQ, shape, dtype)
    if dK is None:
        dK = torch.empty(kv, dtype=dtype, device=device)
    else:
        _check("dK", dK, kv, dtype)
    if dV is None:
        dV = torch.empty(kv, dtype=dtype, device=device)
    else:
        _check("dV", dV, kv, dtype)
    if q_lengths is not None:
        _check_dense("q_lengths", q_lengths, (b,), torch.int32)
        q_lengths = q_lengths.data_ptr()
    if k_lengths is not None:
        _check_dense("k_lengths", k_lengths, (b,), torch.int32)
        k_lengths = k_lengths.data_ptr()
    _call(lib().linformer_softmax_attn_bwd, device,
          (Q.data_ptr(), _strides(Q), K.data_ptr(), _strides(K), V.data_ptr(), _strides(V),
           O.data_ptr(), _strides(O), dO.data_ptr(), _strides(dO), lse.data_ptr(), dQ.data_ptr(),
           _strides(dQ), dK.data_ptr(), _strides(dK), dV.data_ptr(), _strides(dV), q_lengths,
           k_lengths, b, hq, hk, n, m, d, d ** -0.5 if scale is None else scale, 1 if causal else 0,
           _int32("window", window), dtype_code(Q), handle),
          "linformer_softmax_attn_bwd")
    return dQ, dK, dV


def rotary_phase(rot: int, base: float = 10000.0, scaling: int = ROTARY_PLAIN,
                 factor: float = 1.0, original_length: int = 0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, device="cuda", stream=None):
    """The table of `rot / 2` frequencies that rotary() takes (int64, made once and kept)."""
    import torch
    if stream is not None:
        with _current_on(torch.device(device), stream):
            return rotary_phase(rot, base, scaling, factor, original_length, beta_fast, beta_slow,
                                device)
    for name, x in (("rot", rot), ("scaling", scaling), ("original_length", original_length)):
        _int32(name, x)
    phase = torch.empty(max(rot // 2, 1), dtype=torch.int64, device=device)
    handle = _stream_of(phase.device)
    _call(lib().linformer_rotary_phase, phase.device,
          (phase.data_ptr(), rot, base, scaling, factor, original_length, beta_fast, beta_slow, handle),
          "linformer_rotary_phase")
    return phase


def rotary(x, x2=None, phase=None, positions=None, start: int = 0, rot=None,
           layout: int = ROTARY_HALVES, amplitude: float = 1.0, inverse: bool = False, out=None,
           out2=None, stream=None):
    """x [b][h][n][d] (and x2 [b][h2][n][d], or None) turned to their positions; (y, y2) or y.

    positions int32 [b][n], or None for start + row; rot defaults to d.  inverse=True maps
    gradients of the results to gradients of the inputs.  out may be x (in place)."""
    import torch
    if stream is not None:
        with _current_on(x.device, stream):
            return rotary(x, x2, phase, positions, start, rot, layout, amplitude, inverse, out, out2)
    shape, dtype, device = x.shape, x.dtype, x.device
    b, h, n, d = shape
    if rot is None:
        rot = d
    _sizes("x", shape)
    _int32("rot", rot)
    _int32("layout", layout)
    _int32("start", start)
    handle = _stream_of(device, x2, phase, positions, out, out2)
    if phase is None:
        raise ValueError("phase: the table of rotary_phase() is needed")
    _check_dense("phase", phase, (rot // 2,), torch.int64)
    if positions is not None:
        _check_dense("positions", positions, (b, n), torch.int32)
        positions = positions.data_ptr()
    if out is None:
        out = torch.empty_like(x)
    else:
        _check("out", out, shape, dtype)
    px2 = sx2 = py2 = sy2 = None
    h2 = 0
    if x2 is not None:
        h2 = _int32("x2's heads", x2.shape[1])
        _check("x2", x2, (b, h2, n, d), dtype)
        if out2 is None:
            out2 = torch.empty_like(x2)
        else:
            _check("out2", out2, x2.shape, dtype)
        px2, sx2, py2, sy2 = x2.data_ptr(), _strides(x2), out2.data_ptr(), _strides(out2)
    _call(lib().linformer_rotary, device,
          (x.data_ptr(), _strides(x), out.data_ptr(), _strides(out), h, px2, sx2, py2, sy2, h2,
           phase.data_ptr(), positions, start, b, n, d, rot, layout, amplitude,
           1 if inverse else 0, dtype_code(x), handle),
          "linformer_rotary")
    return out if x2 is None else (out, out2)


# --- a paged key/value cache ----------------------------------------------------------------
#
# k_cache and v_cache [pages][hk][page][d] (any strides: a cache laid out [pages][page][hk][d] is
# its transpose(1, 2), one with keys and values side by side two slices), table int32 [b][width]:
# the pages of each sequence in order.  A page, path or tree on the device that is not there is
# recorded in the device status word, as a wait that ran out is.

# (torch's types are passed along: an import in each helper costs as much as its check; arguments go in
# one block: thirty of them one by one cost more than the call's launch)

_PACKED_APPEND, _PACKED_KEEP, _PACKED_ATTN, _PACKED_TREE = 0, 1, 2, 3
_append_words = struct.Struct("=39qd2q")
_keep_words = struct.Struct("=21q")
_attn_words = struct.Struct("=28qd4q")
_tree_words = struct.Struct("=29qd2q")


def _rows(x):
    """A tensor's address and (batch or page, head, row) strides."""
    batch, head, row, last = x.stride()
    if last != 1 and not x.is_contiguous():
        raise ValueError("the last dimension has to be contiguous")
    return x.data_ptr(), batch, head, row

def _check_cache(k_cache, v_cache, table, b, hk, d, dtype, int32):
    """(pages, page, width) of a cache that fits the call's tensors."""
    shape = k_cache.shape
    pages, heads, page, dim = shape
    if heads != hk or dim != d or k_cache.dtype != dtype:
        _check("k_cache", k_cache, (pages, hk, page, d), dtype)
    if v_cache.shape != shape or v_cache.dtype != dtype:
        _check("v_cache", v_cache, shape, dtype)
    entries = table.shape
    width = entries[-1]
    if entries != (b, width) or table.dtype != int32 or not table.is_contiguous():
        _check_dense("table", table, (b, width), int32)
    # (a size past 32 bits comes with as many elements, or with a size of zero, which is refused)
    if k_cache.numel() > 0x7fffffff or width > 0x7fffffff:
        _sizes("k_cache", shape)
        _sizes("table", table.shape)
    return pages, page, width


def _int32s(name, x, shape, int32):
    """Address of a dense int32 tensor, 0 for None."""
    if x is None:
        return 0
    if x.shape != shape or x.dtype != int32 or not x.is_contiguous():
        _check_dense(name, x, shape, int32)
    return x.data_ptr()


def cache_append(K, V, k_cache, v_cache, table, starts, counts=None, Q=None, phase=None,
                 positions=None, rot=None, layout: int = ROTARY_HALVES, amplitude: float = 1.0,
                 out=None, stream=None):
    """Rows i < counts[b] (None: all) of K and V [b][hk][n][d] into rows starts[b] + i of the
    cache, keys turned to their positions where phase is given (the table of rotary_phase();
    positions int32 [b][n], or None for starts[b] + i).  Q [b][hq][n][d], at the same positions, is
    turned in the same call: returns it (in `out`, which may be Q), or None without Q."""
    import torch
    if stream is not None:
        with _current_on(K.device, stream):
            return cache_append(K, V, k_cache, v_cache, table, starts, counts, Q, phase, positions,
                                rot, layout, amplitude, out)
    shape, dtype, device, int32 = K.shape, K.dtype, K.device, torch.int32
    b, hk, n, d = shape
    if K.numel() > 0x7fffffff:
        _sizes("K", shape)
    handle = _stream_of(device, V, k_cache, v_cache, table, starts, counts, Q, phase, positions, out)
    if V.shape != shape or V.dtype != dtype:
        _check("V", V, shape, dtype)
    pages, page, width = _check_cache(k_cache, v_cache, table, b, hk, d, dtype, int32)
    if phase is not None:
        rot = d if rot is None else _int32("rot", rot)
        _int32("layout", layout)
        if phase.shape != (rot // 2,) or phase.dtype != torch.int64 or not phase.is_contiguous():
            _check_dense("phase", phase, (rot // 2,), torch.int64)
        phase = phase.data_ptr()
    elif Q is not None or positions is not None or rot is not None:
        raise ValueError("phase: the table of rotary_phase() is needed to turn keys and queries")
    else:
        rot = phase = 0
    hq, turned_rows = 0, (0,) * 8
    if Q is not None:
        turned = Q.shape
        hq = turned[1]
        if turned != (b, hq, n, d) or Q.dtype != dtype:
            _check("Q", Q, (b, hq, n, d), dtype)
        _int32("Q's heads", hq)
        if out is None:
            out = torch.empty_like(Q)
        elif out.shape != turned or out.dtype != dtype:
            _check("out", out, turned, dtype)
        turned_rows = _rows(Q) + _rows(out)
    elif out is not None:
        raise ValueError("out: Q is needed")
    words = _append_words.pack(
        *_rows(K), *_rows(V), *_rows(k_cache), *_rows(v_cache), *turned_rows, table.data_ptr(),
        _int32s("starts", starts, (b,), int32), _int32s("counts", counts, (b,), int32), phase,
        _int32s("positions", positions, (b, n), int32), b, hq, hk, n, d, pages, page, width, rot, layout,
        amplitude, BF16 if dtype is torch.bfloat16 else dtype_code(K), handle)
    _call(lib().linformer_cache_packed, device, (_PACKED_APPEND, words, 42), "linformer_cache_append")
    return out


def cache_keep(k_cache, v_cache, table, starts, path, counts=None, stream=None):
    """Moves the accepted rows of each sequence's tree, starts[b] + path[b][i], to starts[b] + i,
    for i < counts[b] (None: all of path int32 [b][m]), path[b][i] >= i."""
    import torch
    if stream is not None:
        with _current_on(k_cache.device, stream):
            return cache_keep(k_cache, v_cache, table, starts, path, counts)
    device, dtype, int32 = k_cache.device, k_cache.dtype, torch.int32
    _, hk, _, d = k_cache.shape
    b, m = path.shape
    if path.numel() > 0x7fffffff:
        _sizes("path", path.shape)
    handle = _stream_of(device, v_cache, table, starts, path, counts)
    pages, page, width = _check_cache(k_cache, v_cache, table, b, hk, d, dtype, int32)
    words = _keep_words.pack(
        *_rows(k_cache), *_rows(v_cache), table.data_ptr(), _int32s("starts", starts, (b,), int32),
        _int32s("path", path, (b, m), int32), _int32s("counts", counts, (b,), int32), b, hk, m, d, pages, page, width,
        BF16 if dtype is torch.bfloat16 else dtype_code(k_cache), handle)
    _call(lib().linformer_cache_packed, device, (_PACKED_KEEP, words, 21), "linformer_cache_keep")


def _over_pages(Q, k_cache, v_cache, table, k_lengths, q_lengths, scale, out, lse, mask, masks,
                call, block, name):
    """What paged_attention and tree_attention share; masks: the integers between scale and
    dtype; block: the form of the packed call's arguments."""
    import torch
    shape, dtype, device, int32 = Q.shape, Q.dtype, Q.device, torch.int32
    b, hq, n, d = shape
    if Q.numel() > 0x7fffffff:
        _sizes("Q", shape)
    handle = _stream_of(device, k_cache, v_cache, table, k_lengths, q_lengths, out, lse, mask)
    hk = _int32("k_cache's heads", k_cache.shape[1])
    pages, page, width = _check_cache(k_cache, v_cache, table, b, hk, d, dtype, int32)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    elif out.shape != shape or out.dtype != dtype:
        _check("out", out, shape, dtype)
    if lse is None:
        lse = torch.empty((b, hq, n), dtype=torch.float32, device=device)
    elif lse.shape != (b, hq, n) or lse.dtype != torch.float32 or not lse.is_contiguous():
        _check_dense("lse", lse, (b, hq, n), torch.float32)
    if mask is not None:
        words = (b, n, (n + 63) // 64)
        if mask.shape != words or mask.dtype != torch.int64 or not mask.is_contiguous():
            _check_dense("mask", mask, words, torch.int64)
        mask = (mask.data_ptr(),)
    if k_lengths is None:
        raise ValueError("k_lengths: the rows of each sequence are needed")
    words = block.pack(
        *_rows(Q), *_rows(k_cache), *_rows(v_cache), *_rows(out), lse.data_ptr(), table.data_ptr(),
        _int32s("k_lengths", k_lengths, (b,), int32), _int32s("q_lengths", q_lengths, (b,), int32),
        *(mask or ()), b, hq, hk, n, d, pages, page, width, d ** -0.5 if scale is None else scale, *masks,
        BF16 if dtype is torch.bfloat16 else dtype_code(Q), handle)
    _call(lib().linformer_cache_packed, device, (call, words, block.size // 8), name)
    return out, lse


def paged_attention(Q, k_cache, v_cache, table, k_lengths, q_lengths=None, causal: bool = True,
                    window: int = 0, scale=None, out=None, lse=None, stream=None):
    """(O, lse) of the exact attention of Q [b][hq][n][d], the last n (or q_lengths[b]) tokens of
    each sequence, over the k_lengths[b] (int32 [b]) rows that it has in the cache: single tokens, a
    few, or a chunk of a prompt.  Masks and results are softmax_attention's."""
    if stream is not None:
        with _current_on(Q.device, stream):
            return paged_attention(Q, k_cache, v_cache, table, k_lengths, q_lengths, causal, window,
                                   scale, out, lse)
    return _over_pages(Q, k_cache, v_cache, table, k_lengths, q_lengths, scale, out, lse, None,
                       (1 if causal else 0, _int32("window", window)),
                       _PACKED_ATTN, _attn_words, "linformer_paged_attn_fwd")


def tree_attention(Q, k_cache, v_cache, table, k_lengths, mask, q_lengths=None, scale=None,
                   out=None, lse=None, stream=None):
    """(O, lse) as paged_attention, for a tree of drafted tokens: query i sees every row before the
    tree, and the nodes of the tree whose bits are set in mask[b][i] (int64 [b][n][ceil(n / 64)],
    tree_mask())."""
    if stream is not None:
        with _current_on(Q.device, stream):
            return tree_attention(Q, k_cache, v_cache, table, k_lengths, mask, q_lengths, scale, out,
                                  lse)
    if mask is None:
        raise ValueError("mask: the words of tree_mask() are needed")
    return _over_pages(Q, k_cache, v_cache, table, k_lengths, q_lengths, scale, out, lse, mask, (),
                       _PACKED_TREE, _tree_words, "linformer_tree_attn_fwd")


def tree_mask(parents, out=None, stream=None):
    """int64 [b][n][ceil(n / 64)]: bit j of row i where j is i or one of its ancestors, of trees
    given by parents int32 [b][n] (-1 for a root, else a node before)."""
    import torch
    if stream is not None:
        with _current_on(parents.device, stream):
            return tree_mask(parents, out)
    entries, device = parents.shape, parents.device
    b, n = entries
    if parents.numel() > 0x7fffffff:
        _sizes("parents", entries)
    handle = _stream_of(device, out)
    if parents.dtype != torch.int32 or not parents.is_contiguous():
        _check_dense("parents", parents, entries, torch.int32)
    shape = (b, n, (n + 63) // 64)
    if out is None:
        out = torch.empty(shape, dtype=torch.int64, device=device)
    else:
        _check_dense("out", out, shape, torch.int64)
    _call(lib().linformer_tree_mask, device,
          (parents.data_ptr(), out.data_ptr(), b, n, handle), "linformer_tree_mask")
    return out
