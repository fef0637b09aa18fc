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
import threading

from . import build as _build

PER_HEAD, KV, HEADWISE, LAYERWISE = 0, 1, 2, 3
F32, BF16, BF16_F32OUT = 0, 1, 2
PATH_SIMT, PATH_TENSOR = 0, 1
KERNEL_COUNT = 10
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

_stride_table = {}  # (batch, head, row) strides -> int64[3]


def _strides(x):
    """Address of the tensor's batch, head and row strides (None: dense)."""
    if x.is_contiguous():
        return None
    key = x.stride()
    arr = _stride_table.get(key)
    if arr is None:
        if key[3] != 1:
            raise ValueError("the last dimension has to be contiguous")
        if len(_stride_table) >= 4096:
            _stride_table.clear()
        arr = _stride_table[key] = (ctypes.c_int64 * 3)(*key[:3])
    return arr


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
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {device} and {t.device}")
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(device.index)
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
