"""Thin Python binding of the kvq C ABI (``include/kvq.h``).

Argument marshalling only: every step of the path runs in the CUDA library
``_lib/libkvq.so`` (built by ``build_native.build()``).  There is no Python
or CPU fallback -- if the library is missing, ``load()`` raises.

Functions take either torch tensors (device memory, the current torch stream
by default) or raw integer addresses.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional, Sequence

__all__ = [
    "KvqError", "load", "lib_path", "cache_layout", "quantize_append", "decode_attention",
    "kvq_cache_layout", "kvq_quantize_append", "kvq_decode_attention", "KVQ_MAX_HEADS",
    "decode_attention_static_ws", "kvq_decode_attention_static_ws", "STATIC_WS_BYTES",
    "decode_step", "kvq_decode_step", "decode_attention_ragged", "kvq_decode_attention_ragged",
    "decode_step_ragged", "kvq_decode_step_ragged", "sensitivity_probe", "kvq_sensitivity_probe",
    "probe_workspace_bytes", "kvq_probe_workspace_bytes", "decode_attention_mq",
    "kvq_decode_attention_mq", "decode_mq_workspace_bytes", "kvq_decode_mq_workspace_bytes",
    "KVQ_MAX_QUERY_TOKENS", "workspace_status", "kvq_workspace_status", "set_wait_limits",
    "kvq_set_wait_limits", "set_cache_preload", "kvq_set_cache_preload", "STATUS_TILE_WAIT", "STATUS_PEER_WAIT", "STATUS_COUNTER",
    "decode_tree_workspace_bytes", "kvq_decode_tree_workspace_bytes", "decode_attention_tree",
    "kvq_decode_attention_tree", "tree_commit", "kvq_tree_commit", "attention_mass", "kvq_attention_mass",
    "cache_evict", "kvq_cache_evict", "RopeDesc", "rope_desc", "norm_rope", "kvq_norm_rope", "tree_verify",
    "kvq_tree_verify", "decode_attention_window", "kvq_decode_attention_window", "KVQ_MAX_ROPE_AXES",
    "SEG_K_CODES", "SEG_K_SZ", "SEG_V_CODES", "SEG_V_SZ", "SEG_PROT_K", "SEG_PROT_V",
    "SEG_TEXT_K", "SEG_TEXT_V", "EXPORTED_SYMBOLS",
]

KVQ_MAX_HEADS = 128
KVQ_MAX_QUERY_TOKENS = 64
KVQ_MAX_ROPE_AXES = 4
KVQ_NSEG = 8
(SEG_K_CODES, SEG_K_SZ, SEG_V_CODES, SEG_V_SZ, SEG_PROT_K, SEG_PROT_V, SEG_TEXT_K,
 SEG_TEXT_V) = range(8)
STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_UNSUPPORTED",
          3: "KVQ_ERR_CAPACITY", 4: "KVQ_ERR_CUDA"}
EXPORTED_SYMBOLS = ["kvq_cache_layout", "kvq_quantize_append", "kvq_decode_attention",
                    "kvq_decode_step", "kvq_decode_attention_ragged", "kvq_decode_step_ragged",
                    "kvq_sensitivity_probe", "kvq_probe_workspace_bytes", "kvq_decode_attention_mq",
                    "kvq_decode_mq_workspace_bytes",
                    "kvq_decode_attention_static_ws", "kvq_workspace_status", "kvq_set_wait_limits",
                    "kvq_set_cache_preload", "kvq_decode_tree_workspace_bytes", "kvq_decode_attention_tree",
                    "kvq_tree_commit", "kvq_attention_mass", "kvq_cache_evict",
                    "kvq_norm_rope", "kvq_tree_verify", "kvq_decode_attention_window",
                    "kvq_last_cuda_error", "kvq_status_string"]
STATUS_TILE_WAIT, STATUS_PEER_WAIT, STATUS_COUNTER = 1, 2, 4  # KVQ_STATUS_* bits
STATIC_WS_BYTES = 16 * 1024 * 1024  # KVQ_STATIC_WS_BYTES

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "_lib", "libkvq.so")


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = f"{what}: {STATUS.get(status, status)}"
        self.cuda_error = 0
        if status == 4 and _lib is not None:
            self.cuda_error = int(_lib.kvq_last_cuda_error())
            msg += f" (cudaError {self.cuda_error})"
        super().__init__(msg)
        self.status = status


class LayoutDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("T_cap", ctypes.c_int32), ("vis_start", ctypes.c_int32),
                ("vis_end", ctypes.c_int32), ("k_bits", ctypes.c_int32),
                ("v_bits", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("protected_heads", ctypes.c_uint8 * KVQ_MAX_HEADS)]


class Layout(ctypes.Structure):
    _fields_ = [("d", LayoutDesc), ("g", ctypes.c_int32), ("n_prot", ctypes.c_int32),
                ("n_packed", ctypes.c_int32), ("Tv", ctypes.c_int32), ("Tv_pad", ctypes.c_int32),
                ("T_text", ctypes.c_int32),
                ("units", ctypes.c_int32),
                ("slot", ctypes.c_int32 * KVQ_MAX_HEADS),
                ("prot_head", ctypes.c_uint8 * KVQ_MAX_HEADS),
                ("packed_head", ctypes.c_uint8 * KVQ_MAX_HEADS),
                ("row_bytes", ctypes.c_int64 * KVQ_NSEG), ("off", ctypes.c_int64 * KVQ_NSEG),
                ("bytes", ctypes.c_int64 * KVQ_NSEG), ("total_bytes", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64), ("eff_bits_k", ctypes.c_double),
                ("eff_bits_v", ctypes.c_double), ("n_konly", ctypes.c_int32),
                ("konly_head", ctypes.c_uint8 * KVQ_MAX_HEADS)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("axis", ctypes.c_uint8 * 64)]


# kvq_rows as bytes (data, stride_b, stride_h, stride_t): a Structure takes
# several times as long to make, and norm_rope needs four a call
_ROWS = struct.Struct("=Qqqq").pack


_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"kvq native library missing at {path}; build it with "
                           "bit_mixed_precision_kvq_gb300.build_native.build()")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
    lib.kvq_cache_layout.argtypes = [ctypes.POINTER(LayoutDesc), ctypes.POINTER(Layout)]
    lib.kvq_cache_layout.restype = ctypes.c_int
    lib.kvq_quantize_append.argtypes = [ctypes.POINTER(Layout), P, P, P, i64, i64, i64, i32, i32, P]
    lib.kvq_quantize_append.restype = ctypes.c_int
    lib.kvq_decode_attention.argtypes = [ctypes.POINTER(Layout), P, P, i32, f32, P, P, P, sz, P]
    lib.kvq_decode_attention.restype = ctypes.c_int
    lib.kvq_decode_step.argtypes = [ctypes.POINTER(Layout), P, P, P, P, i32, f32, P, P, P, sz, P]
    lib.kvq_decode_step.restype = ctypes.c_int
    lib.kvq_decode_attention_ragged.argtypes = [ctypes.POINTER(Layout), P, P, P, i32, f32, P, P, P, sz, P]
    lib.kvq_decode_attention_ragged.restype = ctypes.c_int
    lib.kvq_decode_step_ragged.argtypes = [ctypes.POINTER(Layout), P, P, P, P, P, i32, f32, P, P, P, sz,
                                           P]
    lib.kvq_decode_step_ragged.restype = ctypes.c_int
    lib.kvq_decode_mq_workspace_bytes.argtypes = [ctypes.POINTER(Layout), i32]
    lib.kvq_decode_mq_workspace_bytes.restype = sz
    lib.kvq_decode_attention_mq.argtypes = [ctypes.POINTER(Layout), P, P, i32, i32, f32, P, P, P, sz, P]
    lib.kvq_decode_attention_mq.restype = ctypes.c_int
    lib.kvq_probe_workspace_bytes.argtypes = [ctypes.POINTER(Layout), i32]
    lib.kvq_probe_workspace_bytes.restype = sz
    lib.kvq_sensitivity_probe.argtypes = [ctypes.POINTER(Layout), P, P, P, P, i64, i64, i64, i32, f32, P,
                                          i32, P, P, sz, P]
    lib.kvq_sensitivity_probe.restype = ctypes.c_int
    lib.kvq_decode_attention_static_ws.argtypes = [ctypes.POINTER(Layout), P, P, i32, f32, P, P, P]
    lib.kvq_decode_attention_static_ws.restype = ctypes.c_int
    lib.kvq_workspace_status.argtypes = [P, P, P]
    lib.kvq_workspace_status.restype = ctypes.c_int
    lib.kvq_set_wait_limits.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
    lib.kvq_set_wait_limits.restype = None
    lib.kvq_set_cache_preload.argtypes = [ctypes.c_int32]
    lib.kvq_set_cache_preload.restype = None
    LP = ctypes.POINTER(Layout)
    lib.kvq_decode_tree_workspace_bytes.argtypes = [LP, i32]
    lib.kvq_decode_tree_workspace_bytes.restype = sz
    lib.kvq_decode_attention_tree.argtypes = [LP, P, P, P, P, i64, i64, i64, i32, P, i64, P, i32, f32, P, P, P, sz, P]
    lib.kvq_decode_attention_tree.restype = ctypes.c_int
    lib.kvq_tree_commit.argtypes = [LP, P, P, P, i64, i64, i64, i32, P, i32, P, P, i32, P, P]
    lib.kvq_tree_commit.restype = ctypes.c_int
    lib.kvq_attention_mass.argtypes = [LP, P, P, P, i32, P, i32, P, i32, P, f32, P, f32, P, P]
    lib.kvq_attention_mass.restype = ctypes.c_int
    lib.kvq_cache_evict.argtypes = [LP, P, P, P, i32, LP, P, i32, i32, P, P, P, P]
    lib.kvq_cache_evict.restype = ctypes.c_int
    lib.kvq_norm_rope.argtypes = [LP, ctypes.POINTER(RopeDesc), P, P, i32, P, i64, i64, P, P, P, f32, P, P, P]
    lib.kvq_norm_rope.restype = ctypes.c_int
    lib.kvq_tree_verify.argtypes = [i32, i32, i32, P, i32, i64, i64, P, P, i64, P, i64, i64, P, P, P, P, P, P, P, P, P]
    lib.kvq_tree_verify.restype = ctypes.c_int
    lib.kvq_decode_attention_window.argtypes = [LP, P, P, i32, P, i32, i32, i32, f32, P, P, P]
    lib.kvq_decode_attention_window.restype = ctypes.c_int
    lib.kvq_last_cuda_error.argtypes = []
    lib.kvq_last_cuda_error.restype = ctypes.c_int
    lib.kvq_status_string.argtypes = [ctypes.c_int]
    lib.kvq_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _addr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def cache_layout(B: int, H_q: int, H_kv: int, D: int, T_cap: int, vis_start: int, vis_end: int,
                 k_bits: int, v_bits: int, group_size: int,
                 protected: Sequence[int] = (), k_only: Sequence[int] = ()) -> Layout:
    """kvq_cache_layout: validate the per-layer description and derive the layout.
    ``protected`` lists the KV heads whose visual K and V stay bf16, ``k_only``
    those whose visual K alone stays bf16 (V quantised)."""
    d = LayoutDesc(B, H_q, H_kv, D, T_cap, vis_start, vis_end, k_bits, v_bits, group_size)
    for mode, heads in ((1, protected), (2, k_only)):
        for h in heads:
            if not 0 <= int(h) < KVQ_MAX_HEADS or d.protected_heads[int(h)] != 0:
                raise KvqError(1, "kvq_cache_layout")
            d.protected_heads[int(h)] = mode
    out = Layout()
    st = load().kvq_cache_layout(ctypes.byref(d), ctypes.byref(out))
    if st != 0:
        raise KvqError(st, "kvq_cache_layout")
    return out


def quantize_append(L: Layout, cache, k, v, t0: int, n_tok: Optional[int] = None,
                    strides: Optional[Sequence[int]] = None, stream=None) -> None:
    """kvq_quantize_append: write positions [t0, t0 + n_tok) of K and V
    ([B, H_kv, n_tok, D] bf16 on the device) into the cache."""
    if strides is None:
        if k.stride() != v.stride():
            raise ValueError("k and v must share strides")
        if k.stride(-1) != 1:
            raise ValueError("last dim must be contiguous")
        strides = k.stride()[:3]
        n_tok = k.shape[2] if n_tok is None else n_tok
    st = load().kvq_quantize_append(ctypes.byref(L), _addr(cache), _addr(k), _addr(v),
                                    int(strides[0]), int(strides[1]), int(strides[2]), int(t0),
                                    int(n_tok), _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_quantize_append")


def decode_attention(L: Layout, cache, q, T: int, out, softmax_scale: Optional[float] = None,
                     lse=None, workspace=None, ws_bytes: Optional[int] = None,
                     stream=None) -> None:
    """kvq_decode_attention: out[b, hq] = softmax(scale q . k) v over positions [0, T)."""
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(L.d.D)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().kvq_decode_attention(ctypes.byref(L), _addr(cache), _addr(q), int(T),
                                     float(softmax_scale), _addr(out), _addr(lse),
                                     _addr(workspace), int(ws_bytes), _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_decode_attention")


def decode_step(L: Layout, cache, q, k_new, v_new, t_new: int, out,
                softmax_scale: Optional[float] = None, lse=None, workspace=None,
                ws_bytes: Optional[int] = None, stream=None) -> None:
    """kvq_decode_step: one fused decode step.  Stores the new token's bf16 K/V
    rows ([B, H_kv, D]) at text position t_new and attends q over [0, t_new]
    in one cooperative launch.  The workspace's first 4 bytes must be zero
    before its first use (every call leaves them zero)."""
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(L.d.D)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().kvq_decode_step(ctypes.byref(L), _addr(cache), _addr(q), _addr(k_new),
                                _addr(v_new), int(t_new), float(softmax_scale), _addr(out),
                                _addr(lse), _addr(workspace), int(ws_bytes), _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_decode_step")


def decode_attention_ragged(L: Layout, cache, q, seq_len, T_max: int, out,
                            softmax_scale: Optional[float] = None, lse=None, workspace=None,
                            ws_bytes: Optional[int] = None, stream=None) -> None:
    """kvq_decode_attention_ragged: sequence b attends positions
    [0, seq_len[b]) (seq_len: device int32 [B]; an entry outside [1, T_max]
    marks an inactive sequence, whose outputs are zero and lse -inf)."""
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(L.d.D)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().kvq_decode_attention_ragged(ctypes.byref(L), _addr(cache), _addr(q), _addr(seq_len),
                                            int(T_max), float(softmax_scale), _addr(out), _addr(lse),
                                            _addr(workspace), int(ws_bytes), _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_decode_attention_ragged")


def decode_step_ragged(L: Layout, cache, q, k_new, v_new, t_new, T_max: int, out,
                       softmax_scale: Optional[float] = None, lse=None, workspace=None,
                       ws_bytes: Optional[int] = None, stream=None) -> None:
    """kvq_decode_step_ragged: sequence b stores its row at t_new[b] (device
    int32 [B]) and attends [0, t_new[b]]; an entry outside [0, T_max) or
    inside the visual range marks an inactive sequence (nothing stored,
    outputs zero, lse -inf).  Workspace rules as for decode_step."""
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(L.d.D)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().kvq_decode_step_ragged(ctypes.byref(L), _addr(cache), _addr(q), _addr(k_new),
                                       _addr(v_new), _addr(t_new), int(T_max), float(softmax_scale),
                                       _addr(out), _addr(lse), _addr(workspace), int(ws_bytes),
                                       _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_decode_step_ragged")


def decode_mq_workspace_bytes(L: Layout, n_q: int) -> int:
    """kvq_decode_mq_workspace_bytes: workspace bytes of decode_attention_mq."""
    return int(load().kvq_decode_mq_workspace_bytes(ctypes.byref(L), int(n_q)))


def decode_attention_mq(L: Layout, cache, q, T: int, out, softmax_scale: Optional[float] = None,
                        lse=None, workspace=None, ws_bytes: Optional[int] = None,
                        stream=None) -> None:
    """kvq_decode_attention_mq: q [B, n_q, H_q, D] bf16; token i attends
    positions [0, T - n_q + 1 + i); out [B, n_q, H_q, D], lse [B, n_q, H_q]."""
    n_q = int(q.shape[1])
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(L.d.D)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().kvq_decode_attention_mq(ctypes.byref(L), _addr(cache), _addr(q), n_q, int(T),
                                        float(softmax_scale), _addr(out), _addr(lse),
                                        _addr(workspace), int(ws_bytes), _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_decode_attention_mq")


def probe_workspace_bytes(L: Layout, T: int) -> int:
    """kvq_probe_workspace_bytes: scratch bytes of sensitivity_probe over T positions."""
    return int(load().kvq_probe_workspace_bytes(ctypes.byref(L), int(T)))


def sensitivity_probe(L: Layout, cache, q, k, v, T: int, readout, result,
                      softmax_scale: Optional[float] = None, workspace=None,
                      ws_bytes: Optional[int] = None, strides: Optional[Sequence[int]] = None,
                      stream=None) -> None:
    """kvq_sensitivity_probe: per (b, hq), fp64 (kl_attn, kl_out, err) of
    the cache against the raw rows k, v ([B, H_kv, >= T, D] bf16 on the
    device) into result ([B, H_q, 3] float64); readout [n_out, D] float32."""
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(L.d.D)
    if strides is None:
        if k.stride() != v.stride():
            raise ValueError("k and v must share strides")
        if k.stride(-1) != 1:
            raise ValueError("last dim must be contiguous")
        strides = k.stride()[:3]
    n_out = readout.shape[0] if hasattr(readout, "shape") else 0
    if workspace is None:
        import torch
        workspace = torch.empty(max(1, probe_workspace_bytes(L, T)), dtype=torch.uint8,
                                device=result.device)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    st = load().kvq_sensitivity_probe(ctypes.byref(L), _addr(cache), _addr(q), _addr(k), _addr(v),
                                      int(strides[0]), int(strides[1]), int(strides[2]), int(T),
                                      float(softmax_scale), _addr(readout), int(n_out), _addr(result),
                                      _addr(workspace), int(ws_bytes), _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_sensitivity_probe")


def decode_attention_static_ws(L: Layout, cache, q, T: int, out,
                               softmax_scale: Optional[float] = None, lse=None,
                               stream=None) -> None:
    """kvq_decode_attention_static_ws: same result as decode_attention, for
    callers that may not allocate device memory -- the scratch is a fixed
    array inside the library (STATIC_WS_BYTES per GPU).  Calls on one device
    share that array, so they must not overlap on the GPU."""
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(L.d.D)
    st = load().kvq_decode_attention_static_ws(ctypes.byref(L), _addr(cache), _addr(q), int(T),
                                               float(softmax_scale), _addr(out), _addr(lse),
                                               _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_decode_attention_static_ws")


def _refuse(what: str, x, dtype: str, shape, dev: int) -> None:
    """Why a tensor is not what a call needs."""
    import torch
    if x.dtype != getattr(torch, dtype) or (shape is not None and tuple(x.shape) != shape):
        raise ValueError(f"{what}: {dtype} of shape {shape} expected, got {x.dtype} {tuple(x.shape)}")
    if x.get_device() != dev:
        raise ValueError(f"{what} must be on the current CUDA device")
    raise ValueError(f"{what} must be contiguous")


def _ptr(what: str, x, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of the given type and shape on device
    dev; None and raw addresses pass.  The C call would read anything else as
    something it is not."""
    if x is None:
        return 0
    if x.__class__ is int:
        return x
    if x.dtype is dtype and x.shape == shape and x.is_contiguous() and x.get_device() == dev:
        return x.data_ptr()
    return _refuse(what, x, str(dtype)[6:], shape, dev)


def _cache_ptr(what: str, L: Layout, x, dtype, dev: int) -> int:
    if x.__class__ is int:
        return x
    if x.dtype is dtype and x.is_contiguous() and x.get_device() == dev:
        if x.numel() >= L.total_bytes:
            return x.data_ptr()
        raise ValueError(f"{what}: {L.total_bytes} bytes expected, got {x.numel()}")
    return _refuse(what, x, "uint8", None, dev)


def _i32(what: str, x) -> int:
    """x as the int32 that the C call takes (ctypes would drop higher bits)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{what} must be an int32, got {x}")
    return x


def _workspace(x, ws_bytes, dev: int):
    """Address and size of a workspace: a contiguous tensor on device dev, of
    which ws_bytes may name a part, or a raw address with its size."""
    if x is None or x.__class__ is int:
        return x or 0, int(ws_bytes or 0)
    if x.get_device() != dev:
        raise ValueError("workspace must be on the current CUDA device")
    if not x.is_contiguous():
        raise ValueError("workspace must be contiguous")
    have = x.numel() * x.element_size()
    if ws_bytes is None:
        ws_bytes = have
    elif not 0 <= ws_bytes <= have:
        raise ValueError(f"workspace has {have} bytes, ws_bytes is {ws_bytes}")
    return x.data_ptr(), int(ws_bytes)


def _drafts(k, v, shape, dtype, dev: int):
    """Addresses and strides of the drafted rows ([B, H_kv, n_q, D], last
    dimension contiguous)."""
    for what, x in (("k_draft", k), ("v_draft", v)):
        if not (x.dtype is dtype and x.shape == shape and x.get_device() == dev):
            _refuse(what, x, "bfloat16", shape, dev)
    s = k.stride()
    if s != v.stride():
        raise ValueError("k_draft and v_draft must share strides")
    if s[3] != 1:
        raise ValueError("last dim must be contiguous")
    # a dimension of one row has no stride to speak of
    return (k.data_ptr(), v.data_ptr(), s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0,
            s[2] if shape[2] > 1 else 0)


_raw_stream = None


def _current(stream):
    """(torch, current device, raw stream): the given stream, or the current one."""
    import torch
    global _raw_stream
    if _raw_stream is None:  # the public call builds a Stream object first
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    if stream is None:
        dev = torch.cuda.current_device()
        return torch, dev, _raw_stream(dev)
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -2
    return torch, dev, stream if isinstance(stream, int) else int(stream.cuda_stream)


def decode_tree_workspace_bytes(L: Layout, n_q: int) -> int:
    """kvq_decode_tree_workspace_bytes: workspace bytes of decode_attention_tree."""
    return int(load().kvq_decode_tree_workspace_bytes(ctypes.byref(L), int(n_q)))


def decode_attention_tree(L: Layout, cache, q, k_draft, v_draft, tree_mask, T_ctx: int, out,
                          softmax_scale: Optional[float] = None, lse=None, workspace=None,
                          ws_bytes: Optional[int] = None, seq_len=None, stream=None) -> None:
    """kvq_decode_attention_tree: q [B, n_q, H_q, D] bf16, drafted rows
    k_draft, v_draft [B, H_kv, n_q, D] bf16 (any strides of the first three
    dimensions that are multiples of 8), tree_mask int64 [B, n_q], or [n_q] or
    [1, n_q] for one tree of the whole batch (bit j of entry i: token i sees
    draft j).  Token i attends the cache positions [0, seq_len[b]) ([0, T_ctx)
    without seq_len) and its drafts; out [B, n_q, H_q, D], lse [B, n_q, H_q]."""
    if q.dim() != 4:
        raise ValueError("q must be [B, n_q, H_q, D]")
    torch, dev, st = _current(stream)
    d, bf16 = L.d, torch.bfloat16
    B, n_q, Hq = d.B, q.shape[1], d.H_q
    rows = (B, n_q, Hq, d.D)
    cp, qp = _cache_ptr("cache", L, cache, torch.uint8, dev), _ptr("q", q, bf16, rows, dev)
    kp, vp, sb, sh, sd = _drafts(k_draft, v_draft, (B, d.H_kv, n_q, d.D), bf16, dev)
    shared = tree_mask.dim() == 1 or tree_mask.shape[0] != B
    mask = _ptr("tree_mask", tree_mask, torch.int64,
                ((n_q,) if tree_mask.dim() == 1 else (1, n_q)) if shared else (B, n_q), dev)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d.D)
    wp, ws_bytes = _workspace(workspace, ws_bytes, dev)
    st = load().kvq_decode_attention_tree(
        ctypes.byref(L), cp, qp, kp, vp, sb, sh, sd, n_q, mask, 0 if shared else n_q,
        _ptr("seq_len", seq_len, torch.int32, (B,), dev), _i32("T_ctx", T_ctx), softmax_scale,
        _ptr("out", out, bf16, rows, dev), _ptr("lse", lse, torch.float32, (B, n_q, Hq), dev), wp, ws_bytes, st)
    if st != 0:
        raise KvqError(st, "kvq_decode_attention_tree")


def tree_commit(L: Layout, cache, k_draft, v_draft, path, path_len, T_ctx: int, seq_len=None, new_len=None,
                stream=None) -> None:
    """kvq_tree_commit: cache position seq_len[b] + k (T_ctx + k without
    seq_len) takes drafted row path[b, k] (int32 [B, max_path]) for
    k < path_len[b] (int32 [B]); new_len (int32 [B], other memory than
    seq_len) gets the new lengths, -1 for an inactive sequence."""
    if k_draft.dim() != 4 or path.dim() != 2:
        raise ValueError("k_draft must be [B, H_kv, n_q, D] and path [B, max_path]")
    torch, dev, st = _current(stream)
    d, i32 = L.d, torch.int32
    B, n_q, max_path = d.B, k_draft.shape[2], path.shape[1]
    per_seq = (B,)
    kp, vp, sb, sh, sd = _drafts(k_draft, v_draft, (B, d.H_kv, n_q, d.D), torch.bfloat16, dev)
    st = load().kvq_tree_commit(
        ctypes.byref(L), _cache_ptr("cache", L, cache, torch.uint8, dev), kp, vp, sb, sh, sd, n_q,
        _ptr("path", path, i32, (B, max_path), dev), max_path, _ptr("path_len", path_len, i32, per_seq, dev),
        _ptr("seq_len", seq_len, i32, per_seq, dev), _i32("T_ctx", T_ctx), _ptr("new_len", new_len, i32, per_seq, dev), st)
    if st != 0:
        raise KvqError(st, "kvq_tree_commit")


def attention_mass(L: Layout, cache, q, lse, T: int, mass, mass_in=None, softmax_scale: Optional[float] = None,
                   decay: float = 1.0, seq_len=None, path=None, path_len=None, stream=None) -> None:
    """kvq_attention_mass: mass[b, h, t] = decay * mass_in[b, h, t] + the
    attention weight that the tokens' query heads of h give position t.
    q [B, n_q, H_q, D] bf16 and lse [B, n_q, H_q] (or [B, H_q, D] and
    [B, H_q]) of one attention call; mass and mass_in float32
    [B, H_kv, T_cap] (mass_in: None for zeros, or mass itself); path int32
    [B, max_path] and path_len int32 [B] pick the tokens (all without)."""
    torch, dev, st = _current(stream)
    d, f32, i32 = L.d, torch.float32, torch.int32
    B = d.B
    n_q = q.shape[1] if q.dim() == 4 else 1
    rows = (B, n_q, d.H_q) if q.dim() == 4 else (B, d.H_q)
    acc, per_seq = (B, d.H_kv, d.T_cap), (B,)
    T, max_path = _i32("T", T), 0
    if path is not None:
        max_path = path.shape[1] if path.dim() == 2 else 0
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d.D)
    st = load().kvq_attention_mass(
        ctypes.byref(L), _cache_ptr("cache", L, cache, torch.uint8, dev), _ptr("q", q, torch.bfloat16, rows + (d.D,), dev),
        _ptr("lse", lse, f32, rows, dev), n_q, _ptr("seq_len", seq_len, i32, per_seq, dev), T,
        _ptr("path", path, i32, (B, max_path), dev), max_path, _ptr("path_len", path_len, i32, per_seq, dev), softmax_scale,
        _ptr("mass_in", mass_in, f32, acc, dev), decay, _ptr("mass", mass, f32, acc, dev), st)
    if st != 0:
        raise KvqError(st, "kvq_attention_mass")


def cache_evict(L: Layout, cache, mass, T: int, L_dst: Layout, cache_dst, T_dst: int, keep, n_recent: int = 0,
                mass_dst=None, seq_len=None, new_len=None, stream=None) -> None:
    """kvq_cache_evict: the positions of largest mass (float32
    [B, H_kv, T_cap]) copied from cache (lengths T, or seq_len) into
    cache_dst, whose layout L_dst has a smaller visual block; keep int32
    [B, H_kv, T_dst] gets their source positions, mass_dst float32
    [B, H_kv, T_cap_dst] their masses, new_len int32 [B] the new lengths."""
    torch, dev, st = _current(stream)
    d, f32, i32, u8 = L.d, torch.float32, torch.int32, torch.uint8
    B, H = d.B, d.H_kv
    T, T_dst, n_recent = _i32("T", T), _i32("T_dst", T_dst), _i32("n_recent", n_recent)
    st = load().kvq_cache_evict(
        ctypes.byref(L), _cache_ptr("cache", L, cache, u8, dev), _ptr("mass", mass, f32, (B, H, d.T_cap), dev),
        _ptr("seq_len", seq_len, i32, (B,), dev), T, ctypes.byref(L_dst), _cache_ptr("cache_dst", L_dst, cache_dst, u8, dev),
        T_dst, n_recent, _ptr("keep", keep, i32, (B, H, T_dst), dev),
        _ptr("mass_dst", mass_dst, f32, (B, H, L_dst.d.T_cap), dev), _ptr("new_len", new_len, i32, (B,), dev), st)
    if st != 0:
        raise KvqError(st, "kvq_cache_evict")


def rope_desc(rot_dim: int, axes: Sequence[int], interleaved: bool = False) -> RopeDesc:
    """The rotation of norm_rope: the first rot_dim elements of a head in pairs
    (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved; axes names the
    position axis of each pair ([0] * 16 + [1] * 24 + [2] * 24: time, height
    and width in sections)."""
    axes = [int(x) for x in axes]
    if len(axes) * 2 != rot_dim or not 8 <= rot_dim <= 128 or rot_dim % 8:
        raise ValueError("rot_dim must be a multiple of 8 up to 128, with rot_dim / 2 axes")
    if min(axes) < 0 or max(axes) >= KVQ_MAX_ROPE_AXES:
        raise ValueError(f"axes must lie in [0, {KVQ_MAX_ROPE_AXES})")
    R = RopeDesc(rot_dim, 1 if interleaved else 0, max(axes) + 1)
    for i, x in enumerate(axes):
        R.axis[i] = x
    return R


def _rows(what: str, x, shape, dtype, dev: int):
    """[B, n, H, D] (last dimension contiguous, any other strides) as the C call's rows."""
    if not (x.dtype is dtype and x.shape == shape and x.get_device() == dev):
        _refuse(what, x, "bfloat16", shape, dev)
    sb, st, sh, sd = x.stride()
    if sd != 1:
        raise ValueError("last dim must be contiguous")
    # a dimension of one entry has no stride to speak of
    return _ROWS(x.data_ptr(), sb if shape[0] > 1 else 0, sh if shape[2] > 1 else 0, st if shape[1] > 1 else 0)


def norm_rope(L: Layout, R: RopeDesc, q, k, pos, inv_freq, q_out, k_out, q_weight=None, k_weight=None,
              eps: float = 1e-6, stream=None) -> None:
    """kvq_norm_rope: query heads q [B, n, H_q, D] and key heads k
    [B, n, H_kv, D] (bf16, any strides of the first three dimensions that are
    multiples of 8; either may be None with its output), normed where a weight
    ([D] bf16) is given and rotated by pos (int32 [n_axes, B, n], or
    [n_axes, n] for the whole batch; more axes than R names are left alone) times inv_freq (float32 [rot_dim / 2]),
    into q_out and k_out of the same shapes (they may be q and k themselves)."""
    torch, dev, st = _current(stream)
    d, bf16 = L.d, torch.bfloat16
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (q is None and k is None):
        raise ValueError("q and k (one at least) each come with their output")
    x = (k if q is None else q).shape
    if len(x) != 4:
        raise ValueError("q and k must be [B, n, heads, D]")
    B, n, D = d.B, x[1], d.D
    qi = qo = ki = ko = None
    if q is not None:
        x = (B, n, d.H_q, D)
        qi, qo = _rows("q", q, x, bf16, dev), _rows("q_out", q_out, x, bf16, dev)
    if k is not None:
        x = (B, n, d.H_kv, D)
        ki, ko = _rows("k", k, x, bf16, dev), _rows("k_out", k_out, x, bf16, dev)
    at = pos.shape
    if pos.dtype is not torch.int32 or len(at) not in (2, 3) or at[0] < R.n_axes or at[1:] != ((B, n) if len(at) == 3 else (n,)):
        raise ValueError(f"pos: int32 of shape {(R.n_axes, B, n)} or {(R.n_axes, n)} expected, got {pos.dtype} {tuple(at)}")
    if pos.get_device() != dev:
        raise ValueError("pos must be on the current CUDA device")
    if n == 0:
        return
    if n >> 31:
        raise ValueError(f"n must be an int32, got {n}")
    ps = pos.stride()
    if n > 1 and ps[-1] != 1:
        raise ValueError("last dim must be contiguous")
    fp = _ptr("inv_freq", inv_freq, torch.float32, (R.rot_dim // 2,), dev)
    wq, wk = _ptr("q_weight", q_weight, bf16, (D,), dev), _ptr("k_weight", k_weight, bf16, (D,), dev)
    st = load().kvq_norm_rope(ctypes.byref(L), ctypes.byref(R), qi, ki, n, pos.data_ptr(), ps[0] if at[0] > 1 else 0,
                              ps[1] if len(at) == 3 and B > 1 else 0, fp, wq, wk, eps, qo, ko, st)
    if st != 0:
        raise KvqError(st, "kvq_norm_rope")


def tree_verify(logits, tokens, tree_mask, accept, race, path, path_len, next_token, draft_prob=None, temperature=None,
                tree_len=None, logprob=None, stream=None) -> None:
    """kvq_tree_verify: logits [B, n_q, vocab] (bf16 or float32, last dimension
    contiguous) of the drafted tokens (int32 [B, n_q]; token 0 is the sequence's
    last) and their tree_mask (as in decode_attention_tree) give the accepted
    path (int32 [B, n_q], -1 behind its end), path_len and next_token (int32
    [B]) and logprob (float32 [B, n_q]).  accept float32 [B, n_q] and race
    float32 [B, vocab] are uniform and exponential random numbers; draft_prob
    float32 [B, n_q, vocab] the distributions that siblings were drawn from;
    temperature float32 [B] (0: greedy); tree_len int32 [B] tokens of each tree."""
    torch, dev, st = _current(stream)
    f32, i32 = torch.float32, torch.int32
    if logits.dim() != 3 or (draft_prob is not None and draft_prob.dim() != 3):
        raise ValueError("logits and draft_prob must be [B, n_q, vocab]")
    B, n_q, V = logits.shape
    if (B | n_q | V) >> 31:
        raise ValueError(f"the sizes of logits must be int32, got {(B, n_q, V)}")
    rows, per_seq = (B, n_q), (B,)
    if logits.dtype not in (torch.bfloat16, f32):
        _refuse("logits", logits, "float32", (B, n_q, V), dev)
    at = []
    for what, x in (("logits", logits), ("draft_prob", draft_prob)):
        if x is None:
            at.append((0, 0, 0))
            continue
        if x.shape != (B, n_q, V) or x.get_device() != dev or (x is draft_prob and x.dtype is not f32):
            _refuse(what, x, "float32" if x is draft_prob else str(x.dtype)[6:], (B, n_q, V), dev)
        if V > 1 and x.stride(2) != 1:
            raise ValueError("last dim must be contiguous")
        at.append((x.data_ptr(), x.stride(0) if B > 1 else 0, x.stride(1) if n_q > 1 else 0))
    shared = tree_mask.dim() == 1 or tree_mask.shape[0] != B
    mask = _ptr("tree_mask", tree_mask, torch.int64,
                ((n_q,) if tree_mask.dim() == 1 else (1, n_q)) if shared else (B, n_q), dev)
    st = load().kvq_tree_verify(
        B, n_q, V, at[0][0], 1 if logits.dtype is f32 else 0, at[0][1], at[0][2],
        _ptr("tokens", tokens, i32, rows, dev), mask, 0 if shared else n_q, at[1][0], at[1][1], at[1][2],
        _ptr("accept", accept, f32, rows, dev), _ptr("race", race, f32, (B, V), dev),
        _ptr("temperature", temperature, f32, per_seq, dev), _ptr("tree_len", tree_len, i32, per_seq, dev),
        _ptr("path", path, i32, rows, dev), _ptr("path_len", path_len, i32, per_seq, dev),
        _ptr("next_token", next_token, i32, per_seq, dev), _ptr("logprob", logprob, f32, rows, dev), st)
    if st != 0:
        raise KvqError(st, "kvq_tree_verify")


def decode_attention_window(L: Layout, cache, q, T: int, n_sink: int, window: int, out,
                            softmax_scale: Optional[float] = None, lse=None, seq_len=None, stream=None) -> None:
    """kvq_decode_attention_window: q [B, n_q, H_q, D] bf16 (or [B, H_q, D] for
    one token); token i stands at position len - n_q + i (len: T, or seq_len
    int32 [B]) and attends the first n_sink positions and the window positions
    that end at its own; out like q, lse float32 [B, n_q, H_q] (or [B, H_q])."""
    torch, dev, st = _current(stream)
    d = L.d
    if q.dim() not in (3, 4):
        raise ValueError("q must be [B, n_q, H_q, D] or [B, H_q, D]")
    n_q = q.shape[1] if q.dim() == 4 else 1
    rows = (d.B, n_q, d.H_q) if q.dim() == 4 else (d.B, d.H_q)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d.D)
    st = load().kvq_decode_attention_window(
        ctypes.byref(L), _cache_ptr("cache", L, cache, torch.uint8, dev), _ptr("q", q, torch.bfloat16, rows + (d.D,), dev), n_q,
        _ptr("seq_len", seq_len, torch.int32, (d.B,), dev), _i32("T", T), _i32("n_sink", n_sink), _i32("window", window),
        softmax_scale, _ptr("out", out, torch.bfloat16, rows + (d.D,), dev), _ptr("lse", lse, torch.float32, rows, dev), st)
    if st != 0:
        raise KvqError(st, "kvq_decode_attention_window")


def workspace_status(workspace, stream=None) -> int:
    """kvq_workspace_status: the KVQ_STATUS_* bits OR-ed into the
    workspace's status word (synchronises the stream to read them)."""
    import torch
    host = torch.zeros(1, dtype=torch.int32).pin_memory()
    st = load().kvq_workspace_status(_addr(workspace), _addr(host), _stream(stream))
    if st != 0:
        raise KvqError(st, "kvq_workspace_status")
    s = stream if stream is not None else torch.cuda.current_stream()
    if isinstance(s, int):
        torch.cuda.synchronize()
    else:
        s.synchronize()
    return int(host.item()) & 0xFFFFFFFF


def set_wait_limits(tile_polls: int = 0, peer_polls: int = 0) -> None:
    """kvq_set_wait_limits: bounded-wait limits of later decode calls from
    this host thread (0 = default)."""
    load().kvq_set_wait_limits(int(tile_polls), int(peer_polls))


def set_cache_preload(enable: bool) -> None:
    """kvq_set_cache_preload: later uniform single-query decode calls from
    this host thread copy their first cache tiles before the previous
    kernel in the stream has finished (requires that no kernel outside this
    library writes the cache just before a call)."""
    load().kvq_set_cache_preload(1 if enable else 0)


# Same names as the C entry points.
kvq_cache_layout = cache_layout
kvq_quantize_append = quantize_append
kvq_decode_attention = decode_attention
kvq_decode_attention_static_ws = decode_attention_static_ws
kvq_decode_step = decode_step
kvq_decode_attention_ragged = decode_attention_ragged
kvq_decode_step_ragged = decode_step_ragged
kvq_sensitivity_probe = sensitivity_probe
kvq_decode_attention_mq = decode_attention_mq
kvq_decode_mq_workspace_bytes = decode_mq_workspace_bytes
kvq_probe_workspace_bytes = probe_workspace_bytes
kvq_decode_tree_workspace_bytes = decode_tree_workspace_bytes
kvq_decode_attention_tree = decode_attention_tree
kvq_tree_commit = tree_commit
kvq_attention_mass = attention_mass
kvq_cache_evict = cache_evict
kvq_norm_rope = norm_rope
kvq_tree_verify = tree_verify
kvq_decode_attention_window = decode_attention_window
kvq_workspace_status = workspace_status
kvq_set_wait_limits = set_wait_limits
kvq_set_cache_preload = set_cache_preload
