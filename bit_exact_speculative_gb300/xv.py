"""Python binding of libxv.so: argument marshalling, and checks of the tensors.

Each function has the name of the C entry point it calls (include/xv.h) and
takes torch CUDA tensors (any 2-byte dtype for bf16 data, int32, float32);
every step of the computation runs in the library's kernels.  A missing
library raises at import of the first call: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libxv.so")

vp = ctypes.c_void_p
c_int, c_ll, c_sz, c_float = ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_float


class int_arg:
    """An int argument.  ctypes passes a Python int as a C int by itself; its c_int type would make an
    object of every one first (0.13 us against 0.04)."""
    from_param = staticmethod(operator.index)


long_arg = vp   # a 64-bit integer argument travels like an address, and void* converts it in 0.08 us, c_longlong in 0.13


XV_OK, XV_ERR_ARG, XV_ERR_UNSUPPORTED, XV_ERR_WORKSPACE, XV_ERR_CUDA, XV_ERR_DEVICE_CHECK = 0, -1, -2, -3, -4, -5
XV_GEMM_M_MAX = 64
XV_KMAX = 64
XV_CONV_MAX = 8
XV_TOP_MAX = 32


class XVError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"xv error {code}: {msg}")
        self.code = code


class GdnSteps(ctypes.Structure):
    _fields_ = [("q", vp), ("k", vp), ("v", vp), ("beta", vp), ("gate", vp),
                ("qkv_stride", c_ll), ("gate_stride", c_ll), ("rows_per_seq", c_int)]


class BlockConfig(ctypes.Structure):
    _fields_ = [("hidden", c_int), ("vocab", c_int), ("mlp", c_int), ("n_layers", c_int), ("layer_kind", vp),
                ("gdn_heads", c_int), ("gdn_dk", c_int), ("gdn_dv", c_int),
                ("attn_hq", c_int), ("attn_hkv", c_int), ("attn_hd", c_int), ("rms_eps", c_float),
                ("gdn_qk_heads", c_int), ("gdn_conv", c_int), ("gdn_out_norm", c_int)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("norm1", vp), ("w_in", vp), ("w_out", vp), ("norm2", vp), ("w_gate_up", vp), ("w_down", vp),
                ("conv_w", vp), ("out_norm", vp)]


class BlockWeights(ctypes.Structure):
    _fields_ = [("embed", vp), ("layers", vp), ("final_norm", vp), ("lm_head", vp), ("tiled", c_int)]


class LayerState(ctypes.Structure):
    _fields_ = [("gdn_state", vp), ("gdn_hist", vp * 2), ("gdn_conv_state", vp), ("gdn_conv_out", vp * 2),
                ("k_cache", vp), ("v_cache", vp)]


class KvPages(ctypes.Structure):
    _fields_ = [("page_table", vp), ("page_size", c_int), ("max_pages", c_int), ("n_pages", c_int)]
    _table = None   # the table's tensor, where kv_pages made the struct


class BlockState(ctypes.Structure):
    _fields_ = [("B", c_int), ("kmax", c_int), ("Lmax", c_int), ("ctx_len", vp), ("n_commit", vp),
                ("parity", c_int), ("pending_rows", c_int), ("max_ctx", c_int), ("last_k", c_int), ("layers", vp),
                ("kv_pages", KvPages), ("last_k_seq", vp)]


class QkRope(ctypes.Structure):
    _fields_ = [("q_norm", vp), ("k_norm", vp), ("eps", c_float), ("freq", vp), ("rot", c_int), ("interleaved", c_int)]


class KvQ8(ctypes.Structure):
    _fields_ = [("k", vp), ("v", vp), ("k_scale", vp), ("v_scale", vp)]
    _codes = 0   # entries of the smallest code tensor, where kv_q8 made the struct
    _scales = 0
    _dev = -1
    _keep = None


_lib = None

_SIGS = {
    "xv_abi_version": ([], c_int),
    "xv_last_error": ([], ctypes.c_char_p),
    "xv_device_check": ([vp, ctypes.POINTER(ctypes.c_uint)], c_int),
    "xv_launch_count": ([], ctypes.c_ulonglong),
    "xv_set_overlap": ([c_int], c_int),
    "xv_trace_enable": ([c_int], c_int),
    "xv_trace_disable": ([], c_int),
    "xv_trace_count": ([], c_int),
    "xv_trace_read": ([vp, vp, vp, c_int], c_int),
    "xv_trace_kind_name": ([c_int], ctypes.c_char_p),
    "xv_gemm_workspace_size": ([c_int, c_int, c_int], c_sz),
    "xv_gemm_small_m": ([vp, c_int, vp, vp, c_int, c_int, c_int, c_int, vp, c_sz, vp], c_int),
    "xv_gemm_small_m_f32out": ([vp, c_int, vp, vp, c_int, c_int, c_int, c_int, vp, c_sz, vp], c_int),
    "xv_gemm_splits": ([c_int, c_int], c_int),
    "xv_gemm_small_m_noalloc": ([vp, c_int, vp, vp, c_int, c_int, c_int, c_int, vp], c_int),
    "xv_gemm_tiled_bytes": ([c_int, c_int], c_sz),
    "xv_gemm_tile_weights": ([vp, c_int, c_int, vp, vp], c_int),
    "xv_gemm_small_m_tiled": ([vp, c_int, vp, vp, c_int, c_int, c_int, c_int, vp, c_sz, vp], c_int),
    "xv_gemm_small_m_tiled_f32out": ([vp, c_int, vp, vp, c_int, c_int, c_int, c_int, vp, c_sz, vp], c_int),
    "xv_gemm_tile_gate_up": ([vp, c_int, c_int, vp, vp], c_int),
    "xv_gemm_swiglu_tiled": ([vp, c_int, vp, vp, c_int, c_int, c_int, c_int, vp], c_int),
    "xv_gdn_decode_step": ([vp, ctypes.POINTER(GdnSteps), vp, c_ll, c_int, c_int, c_int, c_int, c_int, vp], c_int),
    "xv_gdn_verify": ([vp, ctypes.POINTER(GdnSteps), vp, c_int, ctypes.POINTER(GdnSteps), c_int, vp, c_ll,
                       c_int, c_int, c_int, c_int, c_int, vp], c_int),
    "xv_gdn_verify_grouped": ([vp, ctypes.POINTER(GdnSteps), vp, c_int, ctypes.POINTER(GdnSteps), c_int, vp, c_ll,
                               c_int, c_int, c_int, c_int, c_int, c_int, vp], c_int),
    "xv_gdn_conv": ([vp, vp, c_ll, c_int, vp, c_int, vp, c_ll, c_int, c_int, vp, c_int, c_int, c_int, vp, c_ll, vp],
                    c_int),
    "xv_gated_norm": ([vp, c_ll, vp, c_ll, vp, c_int, c_int, c_int, c_float, vp, c_ll, vp], c_int),
    "xv_attn_split_begin": ([c_int], c_int),
    "xv_attn_workspace_size": ([c_int, c_int, c_int, c_int, c_int], c_sz),
    "xv_attn_decode_rows": ([vp, c_ll, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_float,
                             vp, c_ll, vp, c_ll, vp, c_sz, vp], c_int),
    "xv_kv_append": ([vp, c_ll, vp, c_int, c_int, c_int, c_int, c_int, vp, vp, vp], c_int),
    "xv_attn_decode_rows_paged": ([vp, c_ll, vp, vp, ctypes.POINTER(KvPages), vp, c_int, c_int, c_int, c_int, c_int,
                                   c_int, c_float, vp, c_ll, vp, c_ll, vp, c_sz, vp], c_int),
    "xv_kv_append_paged": ([vp, c_ll, vp, c_int, c_int, c_int, c_int, ctypes.POINTER(KvPages), vp, vp, vp], c_int),
    "xv_kv_pages_workspace_size": ([c_int], c_sz),
    "xv_kv_pages_update": ([vp, int_arg, int_arg, int_arg, vp, vp, vp, vp, vp, vp, vp, int_arg, vp, vp, vp, int_arg, vp, long_arg,
                            vp], c_int),
    "xv_qk_norm_rope": ([vp, long_arg, vp, long_arg, vp, long_arg, vp, long_arg, ctypes.POINTER(QkRope), vp, vp, int_arg, int_arg, int_arg,
                         int_arg, vp], c_int),
    "xv_qk_norm_rope_append": ([vp, long_arg, vp, long_arg, vp, long_arg, ctypes.POINTER(QkRope), vp, vp, vp, int_arg, int_arg, int_arg,
                                int_arg, int_arg, int_arg, vp, vp, vp], c_int),
    "xv_tree_positions": ([vp, vp, vp, int_arg, int_arg, vp, vp], c_int),
    "xv_attn_tree_workspace_size": ([c_int, c_int, c_int, c_int, c_int], c_sz),
    "xv_attn_tree": ([vp, long_arg, vp, vp, vp, vp, long_arg, vp, vp, int_arg, int_arg, int_arg, int_arg, int_arg, int_arg, int_arg,
                      c_float, vp, long_arg, vp, long_arg, vp, long_arg, vp], c_int),
    "xv_attn_tree_paged": ([vp, long_arg, vp, vp, ctypes.POINTER(KvPages), vp, vp, long_arg, vp, vp, int_arg, int_arg, int_arg, int_arg,
                            int_arg, int_arg, c_float, vp, long_arg, vp, long_arg, vp, long_arg, vp], c_int),
    "xv_tree_accept": ([vp, vp, vp, vp, int_arg, int_arg, vp, vp, vp, vp], c_int),
    "xv_kv_append_path": ([vp, long_arg, vp, vp, vp, int_arg, int_arg, int_arg, int_arg, int_arg, vp, vp, vp], c_int),
    "xv_kv_append_path_paged": ([vp, long_arg, vp, vp, vp, int_arg, int_arg, int_arg, int_arg, ctypes.POINTER(KvPages), vp, vp, vp],
                                c_int),
    "xv_kv_append_q8": ([vp, long_arg, vp, vp, int_arg, int_arg, int_arg, int_arg, int_arg, ctypes.POINTER(KvQ8), vp], c_int),
    "xv_kv_append_q8_paged": ([vp, long_arg, vp, vp, int_arg, int_arg, int_arg, int_arg, ctypes.POINTER(KvPages),
                               ctypes.POINTER(KvQ8), vp], c_int),
    "xv_attn_q8_split_begin": ([c_int], c_int),
    "xv_attn_q8_workspace_size": ([c_int, c_int, c_int, c_int, c_int, c_int, c_int], c_sz),
    "xv_attn_decode_rows_q8": ([vp, long_arg, ctypes.POINTER(KvQ8), vp, vp, int_arg, int_arg, int_arg, int_arg, int_arg, int_arg,
                                int_arg, int_arg, int_arg, c_float, vp, long_arg, vp, long_arg, vp, long_arg, vp], c_int),
    "xv_attn_decode_rows_q8_paged": ([vp, long_arg, ctypes.POINTER(KvQ8), ctypes.POINTER(KvPages), vp, vp, int_arg, int_arg,
                                      int_arg, int_arg, int_arg, int_arg, int_arg, int_arg, c_float, vp, long_arg, vp, long_arg,
                                      vp, long_arg, vp], c_int),
    "xv_logprobs_workspace_size": ([c_int, c_int, c_int], c_sz),
    "xv_logprobs": ([vp, long_arg, vp, vp, int_arg, int_arg, vp, vp, int_arg, vp, vp, vp, long_arg, vp], c_int),
    "xv_logprobs_bf16": ([vp, long_arg, vp, vp, int_arg, int_arg, vp, vp, int_arg, vp, vp, vp, long_arg, vp], c_int),
    "xv_gdn_in_dim": ([ctypes.POINTER(BlockConfig)], c_int),
    "xv_gdn_hist_stride": ([ctypes.POINTER(BlockConfig)], c_int),
    "xv_attn_in_dim": ([ctypes.POINTER(BlockConfig)], c_int),
    "xv_gdn_conv_dim": ([ctypes.POINTER(BlockConfig)], c_int),
    "xv_gdn_conv_stride": ([ctypes.POINTER(BlockConfig)], c_int),
    "xv_block_workspace_size": ([ctypes.POINTER(BlockConfig), c_int, c_int, c_int], c_sz),
    "xv_verify_block": ([ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights), ctypes.POINTER(BlockState),
                         vp, c_int, vp, vp, vp, vp, c_sz, vp], c_int),
    "xv_verify_block_commit_accepted": ([ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights),
                                         ctypes.POINTER(BlockState), vp, c_int, vp, vp, vp, vp, c_sz, vp], c_int),
    "xv_block_step_host": ([ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights), ctypes.POINTER(BlockState),
                            vp, vp, c_int, vp, vp, vp, c_sz, vp], c_int),
    "xv_verify_block_ragged": ([ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights),
                                ctypes.POINTER(BlockState), vp, c_int, vp, vp, vp, vp, vp, c_sz, vp], c_int),
    "xv_block_commit": ([ctypes.POINTER(BlockState), vp, vp], c_int),
    "xv_block_commit_accepted": ([ctypes.POINTER(BlockState), vp, vp], c_int),
    "xv_block_flush": ([ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockState), vp], c_int),
    "xv_block_prefill_workspace_size": ([ctypes.POINTER(BlockConfig), c_int, c_int, c_int], c_sz),
    "xv_block_prefill": ([ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights), ctypes.POINTER(BlockState), vp,
                          c_int, c_int, vp, vp, vp, c_sz, vp], c_int),
}


def lib():
    """The loaded libxv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with bit_exact_speculative_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def _check(code: int):
    if code != XV_OK:
        raise XVError(code, lib().xv_last_error().decode(errors="replace"))


# A call's host time is a few microseconds, of the order of a short kernel's: pointers and streams go
# to ctypes as plain ints (the signatures make them void*), and the current stream is asked for as its
# handle (a torch.cuda.Stream object costs ~3 us; it is asked where this torch has no such function).

def _stream_by_object(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_by_object)
# once a CUDA tensor exists: torch.cuda.current_device() without its check that CUDA is initialised (0.1 us against 0.23)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream


def _row_stride(t: torch.Tensor) -> int:
    s = t.stride()
    assert len(s) >= 2 and s[-1] == 1, "rows must be contiguous"
    return s[0]


# The library sees addresses only: a tensor of another type, layout or size than it takes it for is
# read or written past its end.  These give a tensor's address (_rows: and row stride) once it is what
# the call needs, on the device of the call's first tensor; _on, last, gives the stream, on the device
# that must hold them all.  An attribute of a tensor takes ~0.06 us, so each is read once.

def _refuse(name, t, want):
    raise ValueError(f"{name}: {want} on the call's device needed, got {str(t.dtype)[6:]} {list(t.shape)}, "
                     f"strides {list(t.stride())}, on {t.device}")


def _flat(name, t, n, dev, dtype=torch.int32):
    """n or more contiguous entries."""
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous() or t.get_device() != dev:
        _refuse(name, t, f"{n} contiguous {str(dtype)[6:]}")
    return t.data_ptr()


def _one(name, t, dev):
    """One int32."""
    if t.dtype is not torch.int32 or t.numel() < 1 or t.get_device() != dev:
        _refuse(name, t, "1 int32")
    return t.data_ptr()


# bf16, or its bits; a 16-bit float of the other kind would be read as bf16
_BITS16 = (torch.bfloat16, torch.int16, torch.uint16)


def _flat16(name, t, n, dev):
    """n or more contiguous bf16 values."""
    if t.dtype not in _BITS16 or t.numel() < n or not t.is_contiguous() or t.get_device() != dev:
        _refuse(name, t, f"{n} contiguous bfloat16 values (or their bits)")
    return t.data_ptr()


def _rows(name, t, m, width, dev):
    """m or more rows (the first dimension) of width or more bf16 values."""
    shape, stride = t.shape, t.stride()
    try:
        (have, cols), (step, one) = shape, stride
    except ValueError:   # another number of dimensions: a row's must lie densely
        ok = len(shape) > 2 and shape[0] > 0 and t[0].is_contiguous()
        (have, cols), (step, one) = (shape[0], t[0].numel()) if ok else (0, 0), (stride[0], 1) if ok else (0, 0)
    if have < m or cols < width or one != 1 or t.dtype not in _BITS16 or t.get_device() != dev:
        _refuse(name, t, f"{m} rows of {width} contiguous bfloat16 values (or their bits)")
    return t.data_ptr(), step


def _ws(t, dev):
    if not t.is_contiguous() or t.get_device() != dev:
        _refuse("ws", t, "a contiguous workspace")
    return t.data_ptr()


def _on(dev, stream=None):
    if dev < 0 or dev != _current_device():
        raise ValueError("tensors in the current device's memory needed, got " + ("host memory" if dev < 0 else f"cuda:{dev}"))
    if stream is None:
        return _raw_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream: one of cuda:{dev} needed, got one of {stream.device}")
    return stream.cuda_stream


# ------------------------------------------------------------------ misc

def xv_abi_version() -> int:
    return lib().xv_abi_version()


def xv_device_check(stream=None) -> int:
    code = ctypes.c_uint(0)
    _check(lib().xv_device_check(_stream(stream), ctypes.byref(code)))
    return code.value


def xv_launch_count() -> int:
    return int(lib().xv_launch_count())


def xv_set_overlap(enable: bool):
    _check(lib().xv_set_overlap(int(enable)))


def xv_trace_enable(capacity: int):
    _check(lib().xv_trace_enable(capacity))


def xv_trace_disable():
    _check(lib().xv_trace_disable())


def xv_trace_read():
    """Returns a list of (kind name, milliseconds, algorithmic bytes) for every traced launch."""
    import numpy as np
    n = int(lib().xv_trace_count())
    ms = np.zeros(n, np.float32)
    kind = np.zeros(n, np.int32)
    nb = np.zeros(n, np.int64)
    _check(lib().xv_trace_read(ms.ctypes.data, kind.ctypes.data, nb.ctypes.data, n))
    return [(lib().xv_trace_kind_name(int(k)).decode(), float(t), int(b)) for k, t, b in zip(kind, ms, nb)]


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace tensor of at least nbytes (the library's workspaces start zeroed)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ GEMM

def xv_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().xv_gemm_workspace_size(M, N, K))


def xv_gemm_splits(N: int, K: int) -> int:
    return int(lib().xv_gemm_splits(N, K))


class TiledWeight:
    """A weight [N, K] in the GEMM's tiled layout (see :func:`tile_weight`): ``data`` holds the
    tiled copy, ``shape`` is the logical (N, K); ``gated`` marks a gate/up weight tiled by
    :func:`tile_gate_up`."""

    def __init__(self, data: torch.Tensor, N: int, K: int, gated: bool = False):
        self.data, self.shape, self.gated = data, torch.Size((N, K)), gated

    def data_ptr(self) -> int:
        return self.data.data_ptr()

    @property
    def device(self):
        return self.data.device


def xv_gemm_tiled_bytes(N: int, K: int) -> int:
    return int(lib().xv_gemm_tiled_bytes(N, K))


def tile_weight(W: torch.Tensor, stream=None) -> TiledWeight:
    """The tiled copy of a row-major weight W [N, K] (2-byte dtype), made on the device."""
    N, K = W.shape
    data = torch.empty(xv_gemm_tiled_bytes(N, K) // 2, dtype=W.dtype, device=W.device)
    _check(lib().xv_gemm_tile_weights(_ptr(W), N, K, _ptr(data), _stream(stream)))
    return TiledWeight(data, N, K)


def tile_gate_up(W: torch.Tensor, stream=None) -> TiledWeight:
    """The gated tiled copy of a gate/up weight W [2F, K] (F gate rows, then F up rows)."""
    N, K = W.shape
    data = torch.empty(xv_gemm_tiled_bytes(N, K) // 2, dtype=W.dtype, device=W.device)
    _check(lib().xv_gemm_tile_gate_up(_ptr(W), N // 2, K, _ptr(data), _stream(stream)))
    return TiledWeight(data, N, K, gated=True)


def xv_gemm_swiglu(X, Wgu: TiledWeight, act, stream=None):
    """act [M, F] = bf16(silu(g) u) of the gate/up projection X Wgu^T, in one kernel."""
    assert Wgu.gated, "the weight must come from tile_gate_up"
    M, K = X.shape[0], X.shape[1]
    F = Wgu.shape[0] // 2
    _check(lib().xv_gemm_swiglu_tiled(_ptr(X), _row_stride(X), _ptr(Wgu), _ptr(act), _row_stride(act), M, F, K,
                                      _stream(stream)))
    return act


def xv_gemm_small_m(X, W, Y, ws, stream=None):
    """Y = X W^T; W a row-major tensor [N, K] or a :class:`TiledWeight`."""
    M, K = X.shape[0], X.shape[1]
    N = W.shape[0]
    f32 = Y.dtype == torch.float32
    if isinstance(W, TiledWeight) and W.gated:
        raise ValueError("a gated gate/up weight goes through xv_gemm_swiglu")
    if isinstance(W, TiledWeight):
        fn = lib().xv_gemm_small_m_tiled_f32out if f32 else lib().xv_gemm_small_m_tiled
    else:
        fn = lib().xv_gemm_small_m_f32out if f32 else lib().xv_gemm_small_m
    _check(fn(_ptr(X), _row_stride(X), _ptr(W), _ptr(Y), _row_stride(Y), M, N, K, _ptr(ws),
              0 if ws is None else ws.nbytes, _stream(stream)))
    return Y


def xv_gemm_small_m_noalloc(X, W, Y, stream=None):
    """Same GEMM with the library's own fixed scratch (no workspace argument)."""
    M, K = X.shape[0], X.shape[1]
    _check(lib().xv_gemm_small_m_noalloc(_ptr(X), _row_stride(X), _ptr(W), _ptr(Y), _row_stride(Y), M, W.shape[0], K,
                                         _stream(stream)))
    return Y


# ------------------------------------------------------------------- GDN

def gdn_steps(q, k, v, beta, gate, qkv_stride: int, gate_stride: int, rows_per_seq: int) -> GdnSteps:
    return GdnSteps(q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), gate.data_ptr(),
                    qkv_stride, gate_stride, rows_per_seq)


def xv_gdn_decode_step(state, step: GdnSteps, o, o_stride: int, B, H, dk, dv, qk_l2norm: bool, stream=None):
    _check(lib().xv_gdn_decode_step(_ptr(state), ctypes.byref(step), _ptr(o), o_stride, B, H, dk, dv,
                                    int(qk_l2norm), _stream(stream)))


def xv_gdn_verify(state, pending, n_commit, max_commit: int, draft, k: int, o, o_stride: int, B, H, dk, dv,
                  qk_l2norm: bool, stream=None):
    _check(lib().xv_gdn_verify(_ptr(state), None if pending is None else ctypes.byref(pending), _ptr(n_commit),
                               max_commit, None if draft is None else ctypes.byref(draft), k, _ptr(o), o_stride,
                               B, H, dk, dv, int(qk_l2norm), _stream(stream)))


def xv_gdn_verify_grouped(state, pending, n_commit, max_commit: int, draft, k: int, o, o_stride: int, B, H, Hk, dk,
                          dv, qk_l2norm: bool, stream=None):
    _check(lib().xv_gdn_verify_grouped(_ptr(state), None if pending is None else ctypes.byref(pending), _ptr(n_commit),
                                       max_commit, None if draft is None else ctypes.byref(draft), k, _ptr(o),
                                       o_stride, B, H, Hk, dk, dv, int(qk_l2norm), _stream(stream)))


def xv_gdn_conv(state, pend, pend_stride: int, pend_rows: int, n_commit, max_commit: int, x, x_stride: int,
                x_rows: int, k: int, w, B: int, y, y_stride: int, stream=None):
    """state [B, Kc-1, C], w [C, Kc] (2-byte dtypes; w may be None when k = 0); see the C header
    for the rows."""
    C, Kc = state.shape[-1], state.shape[-2] + 1
    _check(lib().xv_gdn_conv(_ptr(state), _ptr(pend), pend_stride, pend_rows, _ptr(n_commit), max_commit, _ptr(x),
                             x_stride, x_rows, k, _ptr(w), C, Kc, B, _ptr(y), y_stride, _stream(stream)))


def xv_gated_norm(o, o_stride: int, z, z_stride: int, w, M: int, H: int, dv: int, eps: float, y, y_stride: int,
                  stream=None):
    _check(lib().xv_gated_norm(_ptr(o), o_stride, _ptr(z), z_stride, _ptr(w), M, H, dv, float(eps), _ptr(y),
                               y_stride, _stream(stream)))


# ------------------------------------------------------------- attention

def xv_attn_split_begin(s: int) -> int:
    """First position of attention split s (fixed absolute boundaries)."""
    return int(lib().xv_attn_split_begin(s))


def xv_attn_workspace_size(B, R, Hq, hd, max_ctx) -> int:
    return int(lib().xv_attn_workspace_size(B, R, Hq, hd, max_ctx))


def xv_attn_decode_rows(q, q_stride, kc, vc, ctx_len, R, B, Hq, Hkv, hd, Lmax, max_ctx, scale, out, out_stride, ws,
                        gate=None, gate_stride=0, stream=None):
    _check(lib().xv_attn_decode_rows(_ptr(q), q_stride, _ptr(kc), _ptr(vc), _ptr(ctx_len), R, B, Hq, Hkv, hd, Lmax,
                                     max_ctx, float(scale), _ptr(gate), gate_stride, _ptr(out), out_stride, _ptr(ws),
                                     ws.nbytes, _stream(stream)))


def xv_kv_append(kv_src, src_stride, ctx_len, R, B, Hkv, hd, Lmax, kc, vc, stream=None):
    _check(lib().xv_kv_append(_ptr(kv_src), src_stride, _ptr(ctx_len), R, B, Hkv, hd, Lmax, _ptr(kc), _ptr(vc),
                              _stream(stream)))


def kv_pages(page_table, page_size: int, n_pages: int) -> KvPages:
    """The page description of a paged KV pool: page_table int32 [B, max_pages], contiguous, on the
    device (kept referenced by the returned struct)."""
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
        raise ValueError(f"page_table: a contiguous int32 [B, max_pages] needed, got {str(page_table.dtype)[6:]} "
                         f"{list(page_table.shape)}, strides {list(page_table.stride())}")
    pages = KvPages(page_table.data_ptr(), int(page_size), int(page_table.shape[1]), int(n_pages))
    pages._table, pages._rows, pages._dev = page_table, page_table.shape[0], page_table.get_device()
    return pages


def _pages_of(pages: KvPages, B, dev):
    """Checks that the table has a row for each of B sequences."""
    if pages._table is not None and (pages._rows < B or pages._dev != dev):
        _refuse("page_table", pages._table, f"{B} rows")


def xv_attn_decode_rows_paged(q, q_stride, kpool, vpool, pages: KvPages, ctx_len, R, B, Hq, Hkv, hd, max_ctx, scale,
                              out, out_stride, ws, gate=None, gate_stride=0, stream=None):
    _check(lib().xv_attn_decode_rows_paged(_ptr(q), q_stride, _ptr(kpool), _ptr(vpool), ctypes.byref(pages),
                                           _ptr(ctx_len), R, B, Hq, Hkv, hd, max_ctx, float(scale), _ptr(gate),
                                           gate_stride, _ptr(out), out_stride, _ptr(ws),
                                           ws.nbytes, _stream(stream)))


def xv_kv_append_paged(kv_src, src_stride, ctx_len, R, B, Hkv, hd, pages: KvPages, kpool, vpool, stream=None):
    _check(lib().xv_kv_append_paged(_ptr(kv_src), src_stride, _ptr(ctx_len), R, B, Hkv, hd, ctypes.byref(pages),
                                    _ptr(kpool), _ptr(vpool), _stream(stream)))


def xv_kv_pages_workspace_size(B: int) -> int:
    return int(lib().xv_kv_pages_workspace_size(B))


def xv_kv_pages_update(pages: KvPages, free_pages, n_free, held, ctx_len, n_new, row_start, pos, slots, ws,
                       n_free_out=None, held_out=None, stream=None):
    """Pages, positions and slots of every request's new rows (the C header has the rules); the
    requests are the entries of ctx_len.  n_free and held are updated in place unless
    n_free_out / held_out are given."""
    B, n_rows, dev = ctx_len.numel(), slots.numel(), ctx_len.get_device()
    _pages_of(pages, B, dev)
    nf, h = _one("n_free", n_free, dev), _flat("held", held, B, dev)
    _check(lib().xv_kv_pages_update(pages.page_table, pages.page_size, pages.max_pages, pages.n_pages,
                                    _flat("free_pages", free_pages, pages.n_pages, dev), nf,
                                    nf if n_free_out is None else _one("n_free_out", n_free_out, dev), h,
                                    h if held_out is None else _flat("held_out", held_out, B, dev),
                                    _flat("ctx_len", ctx_len, B, dev), _flat("n_new", n_new, B, dev), B,
                                    _flat("row_start", row_start, B + 1, dev), _flat("pos", pos, n_rows, dev),
                                    _flat("slots", slots, n_rows, dev, torch.int64), n_rows, _ws(ws, dev), ws.nbytes,
                                    _on(dev, stream)))


# ------------------------------------------------- head norms and rotation

def rope_freqs(rot: int, base: float = 10000.0, scale: float = 1.0, device="cuda") -> torch.Tensor:
    """The frequencies base^(-2i/rot) / scale, i < rot/2, as the library takes them: turns per
    position in 64-bit binary fractions (int64 holding the uint64 bits), the nearest to each."""
    from decimal import Context, Decimal, localcontext
    f = []
    with localcontext(Context(prec=40)):   # a double's 53 bits would be 2^-24 of a turn off at position 2^31
        turns = 1 / (Decimal("6.283185307179586476925286766559005768394") * Decimal(scale))
        step = Decimal(base) ** (Decimal(-2) / max(rot, 1))
        for _ in range(rot // 2):
            f.append(int((turns * 2 ** 64).to_integral_value()) % 2 ** 64)
            turns *= step
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in f], dtype=torch.int64, device=device)


def _qk_rope(q_norm, k_norm, eps, freqs, interleaved, hd, dev):
    return QkRope(None if q_norm is None else _flat16("q_norm", q_norm, hd, dev),
                  None if k_norm is None else _flat16("k_norm", k_norm, hd, dev), eps,
                  None if freqs is None else _flat("freqs", freqs, 0, dev, torch.int64),
                  0 if freqs is None else 2 * freqs.numel(), int(interleaved))


def xv_qk_norm_rope(q, k, pos, Hq, Hkv, hd, q_out, k_out, q_norm=None, k_norm=None, eps=1e-6, freqs=None,
                    interleaved=False, n_rows=None, stream=None):
    """Norms and rotates the heads of q [M, >= Hq*hd] into q_out and of k [M, >= Hkv*hd] into k_out
    (each may be its input); freqs from :func:`rope_freqs` (None: no rotation)."""
    M, dev = q.shape[0], q.get_device()
    r = _qk_rope(q_norm, k_norm, eps, freqs, interleaved, hd, dev)
    a, sa = _rows("q", q, M, Hq * hd, dev)
    b, sb = _rows("q_out", q_out, M, Hq * hd, dev)
    c, sc = _rows("k", k, M, Hkv * hd, dev)
    d, sd = _rows("k_out", k_out, M, Hkv * hd, dev)
    _check(lib().xv_qk_norm_rope(a, sa, b, sb, c, sc, d, sd, ctypes.byref(r), None if pos is None else _flat("pos", pos, M, dev),
                                 None if n_rows is None else _one("n_rows", n_rows, dev), M, Hq, Hkv, hd,
                                 _on(dev, stream)))


def xv_qk_norm_rope_append(q, kv, pos, slots, Hq, Hkv, hd, q_out, kpool, vpool, page_size, n_pages, q_norm=None,
                           k_norm=None, eps=1e-6, freqs=None, interleaved=False, n_rows=None, stream=None):
    """The same with the k heads of kv [M, k | v], normed and rotated, and its v heads written to
    slots (int64 [M]) of the pools."""
    M, dev = q.shape[0], q.get_device()
    r = _qk_rope(q_norm, k_norm, eps, freqs, interleaved, hd, dev)
    size = n_pages * Hkv * page_size * hd
    a, sa = _rows("q", q, M, Hq * hd, dev)
    b, sb = _rows("q_out", q_out, M, Hq * hd, dev)
    c, sc = _rows("kv", kv, M, 2 * Hkv * hd, dev)
    _check(lib().xv_qk_norm_rope_append(a, sa, b, sb, c, sc, ctypes.byref(r),
                                        None if pos is None else _flat("pos", pos, M, dev),
                                        _flat("slots", slots, M, dev, torch.int64),
                                        None if n_rows is None else _one("n_rows", n_rows, dev), M, Hq, Hkv, hd,
                                        page_size, n_pages, _flat16("kpool", kpool, size, dev),
                                        _flat16("vpool", vpool, size, dev), _on(dev, stream)))


# ------------------------------------------------------ a tree of drafts

def _nodes(n_nodes, B, dev):
    return None if n_nodes is None else _flat("n_nodes", n_nodes, B, dev)


def xv_tree_positions(parent, n_nodes, ctx_len, pos, stream=None):
    (B, N), dev = parent.shape, parent.get_device()
    _check(lib().xv_tree_positions(_flat("parent", parent, B * N, dev), _nodes(n_nodes, B, dev),
                                   _flat("ctx_len", ctx_len, B, dev), N, B, _flat("pos", pos, B * N, dev),
                                   _on(dev, stream)))


def xv_attn_tree_workspace_size(B, N, Hq, hd, max_ctx) -> int:
    return int(lib().xv_attn_tree_workspace_size(B, N, Hq, hd, max_ctx))


def xv_attn_tree(q, kc, vc, ctx_len, kv_src, parent, n_nodes, N, B, Hq, Hkv, hd, Lmax, max_ctx, scale, out, ws,
                 gate=None, stream=None):
    """q, kv_src, out and gate are row tensors [B*N, ...] (row strides taken from them)."""
    M, w, size, dev = B * N, Hq * hd, B * Hkv * Lmax * hd, q.get_device()
    a, sa = _rows("q", q, M, w, dev)
    c, sc = _rows("kv_src", kv_src, M, 2 * Hkv * hd, dev)
    g, sg = (None, 0) if gate is None else _rows("gate", gate, M, w, dev)
    o, so = _rows("out", out, M, w, dev)
    _check(lib().xv_attn_tree(a, sa, _flat16("kc", kc, size, dev), _flat16("vc", vc, size, dev),
                              _flat("ctx_len", ctx_len, B, dev), c, sc, _flat("parent", parent, M, dev),
                              _nodes(n_nodes, B, dev), N, B, Hq, Hkv, hd, Lmax, max_ctx, scale, g, sg, o, so, _ws(ws, dev),
                              ws.nbytes, _on(dev, stream)))


def xv_attn_tree_paged(q, kpool, vpool, pages: KvPages, ctx_len, kv_src, parent, n_nodes, N, B, Hq, Hkv, hd, max_ctx,
                       scale, out, ws, gate=None, stream=None):
    M, w, size, dev = B * N, Hq * hd, pages.n_pages * Hkv * pages.page_size * hd, q.get_device()
    _pages_of(pages, B, dev)
    a, sa = _rows("q", q, M, w, dev)
    c, sc = _rows("kv_src", kv_src, M, 2 * Hkv * hd, dev)
    g, sg = (None, 0) if gate is None else _rows("gate", gate, M, w, dev)
    o, so = _rows("out", out, M, w, dev)
    _check(lib().xv_attn_tree_paged(a, sa, _flat16("kpool", kpool, size, dev), _flat16("vpool", vpool, size, dev),
                                    ctypes.byref(pages), _flat("ctx_len", ctx_len, B, dev), c, sc,
                                    _flat("parent", parent, M, dev), _nodes(n_nodes, B, dev), N, B, Hq, Hkv, hd, max_ctx,
                                    scale, g, sg, o, so, _ws(ws, dev), ws.nbytes, _on(dev, stream)))


def xv_tree_accept(tokens, parent, n_nodes, argmax, path, n_keep, next_token, stream=None):
    (B, N), dev = parent.shape, parent.get_device()
    _check(lib().xv_tree_accept(_flat("tokens", tokens, B * N, dev), _flat("parent", parent, B * N, dev),
                                _nodes(n_nodes, B, dev), _flat("argmax", argmax, B * N, dev), N, B,
                                _flat("path", path, B * N, dev), _flat("n_keep", n_keep, B, dev),
                                _flat("next_token", next_token, B, dev), _on(dev, stream)))


def xv_kv_append_path(kv_src, path, n_keep, ctx_len, N, B, Hkv, hd, Lmax, kc, vc, stream=None):
    size, dev = B * Hkv * Lmax * hd, kv_src.get_device()
    a, sa = _rows("kv_src", kv_src, B * N, 2 * Hkv * hd, dev)
    _check(lib().xv_kv_append_path(a, sa, _flat("path", path, B * N, dev),
                                   _flat("n_keep", n_keep, B, dev), _flat("ctx_len", ctx_len, B, dev), N, B, Hkv, hd,
                                   Lmax, _flat16("kc", kc, size, dev), _flat16("vc", vc, size, dev), _on(dev, stream)))


def xv_kv_append_path_paged(kv_src, path, n_keep, ctx_len, N, B, Hkv, hd, pages: KvPages, kpool, vpool, stream=None):
    size, dev = pages.n_pages * Hkv * pages.page_size * hd, kv_src.get_device()
    _pages_of(pages, B, dev)
    a, sa = _rows("kv_src", kv_src, B * N, 2 * Hkv * hd, dev)
    _check(lib().xv_kv_append_path_paged(a, sa,
                                         _flat("path", path, B * N, dev), _flat("n_keep", n_keep, B, dev),
                                         _flat("ctx_len", ctx_len, B, dev), N, B, Hkv, hd, ctypes.byref(pages),
                                         _flat16("kpool", kpool, size, dev), _flat16("vpool", vpool, size, dev),
                                         _on(dev, stream)))


# ------------------------------------------------- a KV cache held in 8 bits

def kv_q8(k, v, k_scale, v_scale) -> KvQ8:
    """The description of an 8-bit cache: codes k and v (uint8 or float8_e4m3fn, [B, Hkv, Lmax, hd] or
    pools [n_pages, Hkv, page_size, hd]) and their scales (float32, without the last dimension), all
    contiguous on one device (kept referenced by the returned struct)."""
    dev = k.get_device()
    for name, t in (("k", k), ("v", v)):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_contiguous() or t.get_device() != dev:
            _refuse(name, t, "contiguous uint8 or float8_e4m3fn codes")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t.dtype is not torch.float32 or not t.is_contiguous() or t.get_device() != dev:
            _refuse(name, t, "contiguous float32 scales")
    q = KvQ8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())
    q._keep, q._dev = (k, v, k_scale, v_scale), dev
    q._codes, q._scales = min(k.numel(), v.numel()), min(k_scale.numel(), v_scale.numel())
    return q


def _q8(cache: KvQ8, heads, hd, dev):
    """Checks that the cache holds `heads` heads of tokens."""
    if cache._dev != dev or cache._codes < heads * hd or cache._scales < heads:
        raise ValueError(f"cache: {heads} heads of {hd} codes with their scales on the call's device needed, got {cache._codes} "
                         f"codes and {cache._scales} scales on cuda:{cache._dev}")
    return ctypes.byref(cache)


def _counts(n_rows, B, dev):
    return None if n_rows is None else _flat("n_rows", n_rows, B, dev)


def xv_kv_append_q8(kv_src, ctx_len, R, B, Hkv, hd, Lmax, cache: KvQ8, n_rows=None, stream=None):
    """Quantises the rows kv_src [B*R, k | v] into the cache (the C header has the rule)."""
    dev = kv_src.get_device()
    a, sa = _rows("kv_src", kv_src, B * R, 2 * Hkv * hd, dev)
    _check(lib().xv_kv_append_q8(a, sa, _flat("ctx_len", ctx_len, B, dev), _counts(n_rows, B, dev), R, B, Hkv, hd, Lmax,
                                 _q8(cache, B * Hkv * Lmax, hd, dev), _on(dev, stream)))


def xv_kv_append_q8_paged(kv_src, ctx_len, R, B, Hkv, hd, pages: KvPages, cache: KvQ8, n_rows=None, stream=None):
    dev = kv_src.get_device()
    _pages_of(pages, B, dev)
    a, sa = _rows("kv_src", kv_src, B * R, 2 * Hkv * hd, dev)
    _check(lib().xv_kv_append_q8_paged(a, sa, _flat("ctx_len", ctx_len, B, dev), _counts(n_rows, B, dev), R, B, Hkv, hd,
                                       ctypes.byref(pages), _q8(cache, pages.n_pages * Hkv * pages.page_size, hd, dev),
                                       _on(dev, stream)))


def xv_attn_q8_split_begin(s: int) -> int:
    """First position of split s of the 8-bit cache's attention (fixed absolute boundaries)."""
    return int(lib().xv_attn_q8_split_begin(s))


def xv_attn_q8_workspace_size(B, R, Hq, hd, max_ctx, window=0, sinks=0) -> int:
    return int(lib().xv_attn_q8_workspace_size(B, R, Hq, hd, max_ctx, window, sinks))


def xv_attn_decode_rows_q8(q, cache: KvQ8, ctx_len, R, B, Hq, Hkv, hd, Lmax, max_ctx, scale, out, ws, window=0, sinks=0,
                           gate=None, n_rows=None, stream=None):
    """q, out and gate are row tensors [B*R, ...] (row strides taken from them)."""
    M, w, dev = B * R, Hq * hd, q.get_device()
    a, sa = _rows("q", q, M, w, dev)
    g, sg = (None, 0) if gate is None else _rows("gate", gate, M, w, dev)
    o, so = _rows("out", out, M, w, dev)
    _check(lib().xv_attn_decode_rows_q8(a, sa, _q8(cache, B * Hkv * Lmax, hd, dev), _flat("ctx_len", ctx_len, B, dev),
                                        _counts(n_rows, B, dev), R, B, Hq, Hkv, hd, Lmax, max_ctx, window, sinks, scale, g, sg,
                                        o, so, _ws(ws, dev), ws.nbytes, _on(dev, stream)))


def xv_attn_decode_rows_q8_paged(q, cache: KvQ8, pages: KvPages, ctx_len, R, B, Hq, Hkv, hd, max_ctx, scale, out, ws, window=0,
                                 sinks=0, gate=None, n_rows=None, stream=None):
    M, w, dev = B * R, Hq * hd, q.get_device()
    _pages_of(pages, B, dev)
    a, sa = _rows("q", q, M, w, dev)
    g, sg = (None, 0) if gate is None else _rows("gate", gate, M, w, dev)
    o, so = _rows("out", out, M, w, dev)
    _check(lib().xv_attn_decode_rows_q8_paged(a, sa, _q8(cache, pages.n_pages * Hkv * pages.page_size, hd, dev),
                                              ctypes.byref(pages), _flat("ctx_len", ctx_len, B, dev), _counts(n_rows, B, dev), R,
                                              B, Hq, Hkv, hd, max_ctx, window, sinks, scale, g, sg, o, so, _ws(ws, dev),
                                              ws.nbytes, _on(dev, stream)))


# ------------------------------------------------------- scores of logits

def xv_logprobs_workspace_size(M: int, V: int, top: int = 0) -> int:
    return int(lib().xv_logprobs_workspace_size(M, V, top))


def xv_logprobs(logits, tokens, logprob, ws, entropy=None, top_ids=None, top_logprobs=None, n_rows=None, stream=None):
    """Scores of logits [M, V] (float32 or bfloat16, rows contiguous): logprob [M] of tokens [M]
    (int32, -1 for none), entropy [M] and the top alternatives top_ids (int32) and top_logprobs [M, n],
    each where given."""
    (M, V), (ld, one), dev = logits.shape, logits.stride(), logits.get_device()
    f32 = logits.dtype is torch.float32
    if not f32 and logits.dtype is not torch.bfloat16 or one != 1 and V > 1:
        _refuse("logits", logits, "float32 or bfloat16 [M, V] with contiguous rows")
    top = 0
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs: both or neither")
    if top_ids is not None:
        if top_ids.dim() != 2:
            _refuse("top_ids", top_ids, f"[{M}, top] int32")
        top = top_ids.shape[1]
        if top_logprobs.dim() != 2 or top_logprobs.shape[1] != top:   # another width would be another layout of the entries
            _refuse("top_logprobs", top_logprobs, f"[{M}, {top}] float32")
    f = torch.float32
    fn = lib().xv_logprobs if f32 else lib().xv_logprobs_bf16
    _check(fn(logits.data_ptr(), max(ld, V) if M == 1 else ld, _flat("tokens", tokens, M, dev), None if n_rows is None else _one("n_rows", n_rows, dev),
              M, V, _flat("logprob", logprob, M, dev, f), None if entropy is None else _flat("entropy", entropy, M, dev, f), top,
              None if top_ids is None else _flat("top_ids", top_ids, M * top, dev),
              None if top_ids is None else _flat("top_logprobs", top_logprobs, M * top, dev, f), _ws(ws, dev), ws.nbytes,
              _on(dev, stream)))


# ------------------------------------------------------------------ block

class Block:
    """Holds the ctypes structs of one model (config, weights, state) over caller-owned tensors.

    ``cfg`` is a dict (hidden, vocab, mlp, kinds, gdn_heads, gdn_dk, gdn_dv, attn_hq, attn_hkv,
    attn_hd, rms_eps); ``weights`` a dict of device tensors (embed, final_norm, lm_head and per
    layer ``f"{l}.norm1"``, ``.w_in``, ``.w_out``, ``.norm2``, ``.w_gu``, ``.w_down`` and, for complete GDN
    layers, ``.conv_w``, ``.onorm``), where lm_head and the four projections are either all
    row-major tensors or all :class:`TiledWeight`;
    ``state`` a dict (ctx_len, n_commit and per layer ``f"{l}.state"``, ``.hist0``, ``.hist1`` (and
    ``.conv``, ``.cout0``, ``.cout1`` with a convolution) or ``.kc``, ``.vc``).  With ``pages`` (a :class:`KvPages` over ``state["page_table"]``) the
    attention caches are page pools.  Tensors are kept referenced here.
    """

    def __init__(self, cfg: dict, weights: dict, state: dict, B: int, kmax: int, Lmax: int, ctx0: int,
                 pages: KvPages | None = None):
        kinds = list(cfg["kinds"])
        self._kinds = (ctypes.c_int32 * len(kinds))(*kinds)
        self.cfg = BlockConfig(cfg["hidden"], cfg["vocab"], cfg["mlp"], len(kinds),
                               ctypes.cast(self._kinds, vp).value, cfg.get("gdn_heads", 0), cfg.get("gdn_dk", 0),
                               cfg.get("gdn_dv", 0), cfg.get("attn_hq", 0), cfg.get("attn_hkv", 0),
                               cfg.get("attn_hd", 0), float(cfg.get("rms_eps", 1e-6)), cfg.get("gdn_qk_heads", 0),
                               cfg.get("gdn_conv", 0), int(cfg.get("gdn_out_norm", 0)))
        self._keep = [weights, state]
        names = ("norm1", "w_in", "w_out", "norm2", "w_gu", "w_down", "conv_w", "onorm")
        lw = [LayerWeights(*[weights[f"{l}.{n}"].data_ptr() if f"{l}.{n}" in weights else None for n in names])
              for l in range(len(kinds))]
        self._lw = (LayerWeights * len(kinds))(*lw)
        gemm = [weights["lm_head"]] + [weights[f"{l}.{n}"] for l in range(len(kinds))
                                       for n in ("w_in", "w_out", "w_gu", "w_down")]
        tiled = {isinstance(t, TiledWeight) for t in gemm}
        if len(tiled) != 1:
            raise ValueError("the projection weights and the LM head must be all tiled or all row-major")
        if True in tiled and not all(weights[f"{l}.w_gu"].gated for l in range(len(kinds))):
            raise ValueError("with tiled weights every w_gu must come from tile_gate_up")
        self.weights = BlockWeights(weights["embed"].data_ptr(), ctypes.cast(self._lw, vp).value,
                                    weights["final_norm"].data_ptr(), weights["lm_head"].data_ptr(), int(tiled.pop()))
        ls = []
        for l, kd in enumerate(kinds):
            if kd == 0:
                conv = f"{l}.conv" in state
                ls.append(LayerState(state[f"{l}.state"].data_ptr(),
                                     (vp * 2)(state[f"{l}.hist0"].data_ptr(), state[f"{l}.hist1"].data_ptr()),
                                     state[f"{l}.conv"].data_ptr() if conv else None,
                                     (vp * 2)(state[f"{l}.cout0"].data_ptr(), state[f"{l}.cout1"].data_ptr())
                                     if conv else (vp * 2)(None, None), None, None))
            else:
                ls.append(LayerState(None, (vp * 2)(None, None), None, (vp * 2)(None, None), state[f"{l}.kc"].data_ptr(),
                                     state[f"{l}.vc"].data_ptr()))
        self._ls = (LayerState * len(kinds))(*ls)
        self.state = BlockState(B, kmax, Lmax, state["ctx_len"].data_ptr(), state["n_commit"].data_ptr(), 0, kmax,
                                ctx0, 0, ctypes.cast(self._ls, vp).value, pages if pages is not None else KvPages(),
                                None)
        self.ws_bytes = int(lib().xv_block_workspace_size(ctypes.byref(self.cfg), B, kmax, Lmax))
        if self.ws_bytes == 0:
            _check(XV_ERR_ARG)

    def gdn_in_dim(self) -> int:
        return int(lib().xv_gdn_in_dim(ctypes.byref(self.cfg)))

    def attn_in_dim(self) -> int:
        return int(lib().xv_attn_in_dim(ctypes.byref(self.cfg)))

    def gdn_conv_stride(self) -> int:
        return int(lib().xv_gdn_conv_stride(ctypes.byref(self.cfg)))


def xv_verify_block(blk: Block, tokens, k: int, logits, argmax, n_accept, ws, stream=None):
    _check(lib().xv_verify_block(ctypes.byref(blk.cfg), ctypes.byref(blk.weights), ctypes.byref(blk.state),
                                 _ptr(tokens), k, _ptr(logits), _ptr(argmax), _ptr(n_accept), _ptr(ws),
                                 ws.nbytes, _stream(stream)))


def xv_verify_block_commit_accepted(blk: Block, tokens, k: int, logits, argmax, n_accept, ws, stream=None):
    _check(lib().xv_verify_block_commit_accepted(ctypes.byref(blk.cfg), ctypes.byref(blk.weights),
                                                 ctypes.byref(blk.state), _ptr(tokens), k, _ptr(logits), _ptr(argmax),
                                                 _ptr(n_accept), _ptr(ws), ws.nbytes,
                                                 _stream(stream)))


def xv_block_step_host(blk: Block, host_tokens, dev_tokens, k: int, dev_results, host_results, ws, stream=None):
    # the library copies these sizes from and into raw pointers: host buffers too short would be
    # overrun on the host, so their sizes are checked here
    B, kmax = blk.state.B, blk.state.kmax
    for name, t, n, host in (("host_tokens", host_tokens, B * k, True), ("dev_tokens", dev_tokens, B * k, False),
                             ("dev_results", dev_results, B * kmax + B, False),
                             ("host_results", host_results, B * kmax + B, True)):
        if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < n or t.is_cuda == host:
            raise ValueError(f"{name}: {n} contiguous int32 in {'host' if host else 'device'} memory needed")
    _check(lib().xv_block_step_host(ctypes.byref(blk.cfg), ctypes.byref(blk.weights), ctypes.byref(blk.state),
                                    _ptr(host_tokens), _ptr(dev_tokens), k, _ptr(dev_results), _ptr(host_results),
                                    _ptr(ws), ws.nbytes, _stream(stream)))


def xv_verify_block_ragged(blk: Block, tokens, k: int, k_seq, logits, argmax, n_accept, ws, stream=None):
    _check(lib().xv_verify_block_ragged(ctypes.byref(blk.cfg), ctypes.byref(blk.weights), ctypes.byref(blk.state),
                                        _ptr(tokens), k, _ptr(k_seq), _ptr(logits), _ptr(argmax), _ptr(n_accept),
                                        _ptr(ws), ws.nbytes, _stream(stream)))


def xv_block_commit(blk: Block, n_keep, stream=None):
    _check(lib().xv_block_commit(ctypes.byref(blk.state), _ptr(n_keep), _stream(stream)))


def xv_block_commit_accepted(blk: Block, n_accept, stream=None):
    _check(lib().xv_block_commit_accepted(ctypes.byref(blk.state), _ptr(n_accept), _stream(stream)))


def xv_block_prefill(blk: Block, tokens, T: int, chunk: int, last_logits, last_argmax, ws, stream=None):
    _check(lib().xv_block_prefill(ctypes.byref(blk.cfg), ctypes.byref(blk.weights), ctypes.byref(blk.state),
                                  _ptr(tokens), T, chunk, _ptr(last_logits), _ptr(last_argmax), _ptr(ws),
                                  ws.nbytes, _stream(stream)))


def xv_block_flush(blk: Block, stream=None):
    _check(lib().xv_block_flush(ctypes.byref(blk.cfg), ctypes.byref(blk.state), _stream(stream)))
