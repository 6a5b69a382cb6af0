"""Python binding of the ds_moe C ABI (``include/ds_moe.h``).

Argument marshalling only: every step of the layer runs in the CUDA kernels
of ``libds_moe.so``.  PyTorch supplies device memory and streams.  There is
no fallback: if the library has not been built, importing the binding's
functions raises.

Names mirror the C entry points: ``q2k_bytes``, ``expert_bytes``,
``quantize_q2k``, ``dequantize_q2k``, ``workspace_bytes``, ``layer``,
``layer_hostio``, ``stack``, ``sync_status``; and for a serving step around
the layer ``page_map``, ``kv_append``, ``paged_attention``, ``verify_drafts``.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libds_moe.so")

DS_OK, DS_ERR_INVALID_ARG, DS_ERR_UNSUPPORTED = 0, -1, -2
DS_ERR_CUDA, DS_ERR_TIMEOUT, DS_ERR_DEVICE_CHECK = -3, -4, -5
DS_F32, DS_BF16, DS_F16 = 0, 1, 2
DS_Q2_K, DS_Q4_K = 0, 1

SYMBOLS = ["ds_moe_q2k_bytes", "ds_moe_expert_bytes", "ds_moe_quantize_q2k",
           "ds_moe_dequantize_q2k", "ds_moe_workspace_bytes", "ds_moe_layer",
           "ds_moe_layer_hostio", "ds_moe_stack", "ds_moe_sync_status", "ds_moe_version",
           "ds_moe_layer_noalloc", "ds_moe_layer_path", "ds_moe_q4k_bytes",
           "ds_moe_expert_bytes_fmt", "ds_moe_quantize_q4k", "ds_moe_dequantize_q4k",
           "ds_moe_stack_mixed", "ds_moe_layer_resident", "ds_moe_layer_path_resident",
           "ds_moe_cache_create", "ds_moe_cache_destroy", "ds_moe_cache_layer", "ds_moe_cache_record",
           "ds_moe_cache_slot", "ds_moe_cache_stats", "ds_moe_page_map", "ds_moe_kv_append",
           "ds_moe_attention_workspace_bytes", "ds_moe_paged_attention", "ds_moe_attention_path",
           "ds_moe_verify_drafts"]

# ds_moe_layer_path results
PATH_NONE, PATH_STREAM, PATH_DECODE3, PATH_GROUPED_GEMV, PATH_TENSOR_CORE, PATH_BATCHED_DECODE = 0, 1, 2, 3, 4, 5
# ds_moe_attention_path results
ATTN_GENERIC, ATTN_DECODE, ATTN_CHUNK = 0, 1, 2


class DsMoeError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"ds_moe error {code}: {msg}")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("n_embd", ctypes.c_int32), ("n_expert", ctypes.c_int32),
                ("n_ff", ctypes.c_int32), ("n_ff_shared", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("router_dtype", ctypes.c_int32), ("routed_scale", ctypes.c_float),
                ("logit_scale", ctypes.c_float), ("bias_select_only", ctypes.c_int32),
                ("expert_format", ctypes.c_int32)]


class Weights(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("shared_gate", ctypes.c_void_p), ("shared_up", ctypes.c_void_p),
                ("shared_down", ctypes.c_void_p), ("experts", ctypes.c_void_p)]


class Residency(ctypes.Structure):
    _fields_ = [("slot", ctypes.c_void_p), ("cache", ctypes.c_void_p), ("experts_host", ctypes.c_void_p)]


class Debug(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("perm", ctypes.c_void_p)]


class AttnShapeC(ctypes.Structure):
    _fields_ = [("n_head", ctypes.c_int32), ("n_head_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("window", ctypes.c_int32)]


class KVCacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


_lib = None


def lib():
    """The loaded libds_moe.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() "
                               "(or python bit_quantized_routed_router_gb300/build.py)")
        _lib = load(LIB_PATH)
    return _lib


def load(path: str):
    """A build of the library at `path` (ctypes handle with its signatures)."""
    L = ctypes.CDLL(path)
    vp, i64, sz, cp = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_char_p
    L.ds_moe_q2k_bytes.restype = sz
    L.ds_moe_q2k_bytes.argtypes = [i64, i64]
    L.ds_moe_q4k_bytes.restype = sz
    L.ds_moe_q4k_bytes.argtypes = [i64, i64]
    L.ds_moe_expert_bytes.restype = sz
    L.ds_moe_expert_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32]
    L.ds_moe_expert_bytes_fmt.restype = sz
    L.ds_moe_expert_bytes_fmt.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    for f in (L.ds_moe_quantize_q2k, L.ds_moe_dequantize_q2k, L.ds_moe_quantize_q4k,
              L.ds_moe_dequantize_q4k):
        f.restype = ctypes.c_int
        f.argtypes = [vp, i64, i64, vp, vp, cp, sz]
    L.ds_moe_workspace_bytes.restype = ctypes.c_int
    L.ds_moe_workspace_bytes.argtypes = [ctypes.POINTER(Shape), i64, ctypes.POINTER(sz), cp, sz]
    L.ds_moe_layer.restype = ctypes.c_int
    L.ds_moe_layer.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, i64, vp, vp,
                               sz, ctypes.POINTER(Debug), vp, cp, sz]
    L.ds_moe_layer_hostio.restype = ctypes.c_int
    L.ds_moe_layer_hostio.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, i64,
                                      vp, vp, sz, vp, cp, sz]
    L.ds_moe_stack.restype = ctypes.c_int
    L.ds_moe_stack.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), ctypes.c_int32,
                               vp, i64, ctypes.c_float, vp, sz, vp, cp, sz]
    L.ds_moe_stack_mixed.restype = ctypes.c_int
    L.ds_moe_stack_mixed.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp,
                                     ctypes.c_int32, vp, i64, ctypes.c_float, vp, sz, vp, cp, sz]
    L.ds_moe_layer_noalloc.restype = ctypes.c_int
    L.ds_moe_layer_noalloc.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, i64,
                                       vp, vp, cp, sz]
    L.ds_moe_sync_status.restype = ctypes.c_int
    L.ds_moe_sync_status.argtypes = [vp, cp, sz]
    L.ds_moe_version.restype = ctypes.c_char_p
    L.ds_moe_version.argtypes = []
    L.ds_moe_layer_resident.restype = ctypes.c_int
    L.ds_moe_layer_resident.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights),
                                        ctypes.POINTER(Residency), vp, i64, vp, vp, sz,
                                        ctypes.POINTER(Debug), vp, cp, sz]
    L.ds_moe_layer_path_resident.restype = ctypes.c_int
    L.ds_moe_layer_path_resident.argtypes = [ctypes.POINTER(Shape), i64]
    L.ds_moe_cache_create.restype = ctypes.c_int
    L.ds_moe_cache_create.argtypes = [ctypes.POINTER(Shape), ctypes.c_int32, ctypes.POINTER(vp), vp, i64,
                                      vp, ctypes.POINTER(vp), cp, sz]
    L.ds_moe_cache_destroy.restype = None
    L.ds_moe_cache_destroy.argtypes = [vp]
    L.ds_moe_cache_layer.restype = ctypes.c_int
    L.ds_moe_cache_layer.argtypes = [vp, ctypes.c_int32, ctypes.POINTER(Weights), vp, i64, vp, vp, sz, vp,
                                     cp, sz]
    L.ds_moe_cache_record.restype = ctypes.c_int
    L.ds_moe_cache_record.argtypes = [vp, ctypes.c_int32, vp, vp, ctypes.POINTER(ctypes.c_int32)]
    L.ds_moe_cache_slot.restype = ctypes.c_int
    L.ds_moe_cache_slot.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]
    L.ds_moe_cache_stats.restype = ctypes.c_int
    L.ds_moe_cache_stats.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64)]
    i32, ash, kvc = ctypes.c_int32, ctypes.POINTER(AttnShapeC), ctypes.POINTER(KVCacheC)
    L.ds_moe_page_map.restype = ctypes.c_int
    L.ds_moe_page_map.argtypes = [vp, vp, i32, i32, vp, i32, vp, i32, i64, vp, vp, i32, vp, vp, vp, vp, cp, sz]
    L.ds_moe_kv_append.restype = ctypes.c_int
    L.ds_moe_kv_append.argtypes = [ash, kvc, vp, vp, i64, i64, vp, i64, vp, cp, sz]
    L.ds_moe_attention_workspace_bytes.restype = ctypes.c_int
    L.ds_moe_attention_workspace_bytes.argtypes = [ash, i32, i64, i32, ctypes.POINTER(sz), cp, sz]
    L.ds_moe_paged_attention.restype = ctypes.c_int
    L.ds_moe_paged_attention.argtypes = [ash, kvc, vp, i32, i64, vp, i64, i64, vp, vp, i32, i32, vp, i64, vp, vp, sz,
                                         vp, cp, sz]
    L.ds_moe_attention_path.restype = ctypes.c_int
    L.ds_moe_attention_path.argtypes = [ash, kvc, vp, i64, i32]
    L.ds_moe_verify_drafts.restype = ctypes.c_int
    L.ds_moe_verify_drafts.argtypes = [vp, i64, vp, i64, i32, i64, i32, vp, vp, i32, i32, vp, vp, vp, vp, vp, cp, sz]
    return L


_tls = threading.local()


def _call(fn, *args):
    try:
        err = _tls.err
    except AttributeError:  # a message buffer for each thread
        err = _tls.err = ctypes.create_string_buffer(512)
    rc = fn(*args, err, 512)
    if rc != DS_OK:
        raise DsMoeError(rc, err.value.decode(errors="replace"))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream
    global _current_stream
    if _current_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (no stream object is made for its address)
        _current_stream = ((lambda: raw(torch.cuda.current_device())) if raw
                           else (lambda: torch.cuda.current_stream().cuda_stream))
    return _current_stream()


_current_stream = None


@dataclass
class MoEShape:
    n_embd: int
    n_expert: int
    n_ff: int
    n_ff_shared: int
    top_k: int
    x_dtype: int = DS_BF16
    router_dtype: int = DS_BF16
    routed_scale: float = 1.0
    logit_scale: float = 1.0
    bias_select_only: int = 0
    expert_format: int = 0  # DS_Q2_K or DS_Q4_K

    def c(self) -> Shape:
        return Shape(self.n_embd, self.n_expert, self.n_ff, self.n_ff_shared, self.top_k,
                     self.x_dtype, self.router_dtype, self.routed_scale, self.logit_scale,
                     self.bias_select_only, self.expert_format)


@dataclass
class MoEWeights:
    """Device tensors of one layer (see include/ds_moe.h for layouts)."""
    router_w: object
    experts: object
    router_bias: object = None
    shared_gate: object = None
    shared_up: object = None
    shared_down: object = None

    def c(self) -> Weights:
        return Weights(_ptr(self.router_w), _ptr(self.router_bias), _ptr(self.shared_gate),
                       _ptr(self.shared_up), _ptr(self.shared_down), _ptr(self.experts))


def version() -> str:
    return lib().ds_moe_version().decode()


def q2k_bytes(rows: int, in_dim: int) -> int:
    return lib().ds_moe_q2k_bytes(rows, in_dim)


def q4k_bytes(rows: int, in_dim: int) -> int:
    return lib().ds_moe_q4k_bytes(rows, in_dim)


def expert_bytes(n_embd: int, n_ff: int, expert_format: int = 0) -> int:
    return lib().ds_moe_expert_bytes_fmt(expert_format, n_embd, n_ff)


def quantize_q2k(w, out, stream=None):
    """w: fp32 device tensor [rows][in_dim]; out: uint8 device tensor of q2k_bytes."""
    rows, in_dim = w.shape
    _call(lib().ds_moe_quantize_q2k, w.data_ptr(), rows, in_dim, out.data_ptr(), _stream(stream))


def dequantize_q2k(q, rows, in_dim, out, stream=None):
    _call(lib().ds_moe_dequantize_q2k, q.data_ptr(), rows, in_dim, out.data_ptr(), _stream(stream))


def quantize_q4k(w, out, stream=None):
    """w: fp32 device tensor [rows][in_dim]; out: uint8 device tensor of q4k_bytes."""
    rows, in_dim = w.shape
    _call(lib().ds_moe_quantize_q4k, w.data_ptr(), rows, in_dim, out.data_ptr(), _stream(stream))


def dequantize_q4k(q, rows, in_dim, out, stream=None):
    _call(lib().ds_moe_dequantize_q4k, q.data_ptr(), rows, in_dim, out.data_ptr(), _stream(stream))


def layer_path(shape: MoEShape, T: int, x=None) -> int:
    """Which kernels ds_moe_layer runs for T tokens (a PATH_* value)."""
    L = lib()
    L.ds_moe_layer_path.restype = ctypes.c_int
    L.ds_moe_layer_path.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
    sh = shape.c()
    rc = L.ds_moe_layer_path(ctypes.byref(sh), T, _ptr(x) if x is not None else 256)
    if rc < 0:
        raise DsMoeError(rc, "shape rejected")
    return rc


def workspace_bytes(shape: MoEShape, T: int) -> int:
    n = ctypes.c_size_t(0)
    _call(lib().ds_moe_workspace_bytes, ctypes.byref(shape.c()), T, ctypes.byref(n))
    return n.value


def layer(shape: MoEShape, weights: MoEWeights, x, out, workspace, debug: dict | None = None,
          stream=None, T: int | None = None):
    """out[T][D] fp32 = MoE layer of x[T][D] (device tensors)."""
    T = x.shape[0] if T is None else T
    dbg = None
    if debug is not None:
        dbg = ctypes.byref(Debug(*[_ptr(debug.get(n)) for n in
                                   ("logits", "ids", "w", "counts", "offsets", "perm")]))
    _call(lib().ds_moe_layer, ctypes.byref(shape.c()), ctypes.byref(weights.c()), x.data_ptr(), T,
          out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), dbg,
          _stream(stream))


def layer_hostio(shape: MoEShape, weights: MoEWeights, x_host, out_host, workspace, stream=None):
    """Same as layer with x and out in (pinned) host memory; enqueues only."""
    _call(lib().ds_moe_layer_hostio, ctypes.byref(shape.c()), ctypes.byref(weights.c()),
          x_host.data_ptr(), x_host.shape[0], out_host.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), _stream(stream))


def layer_noalloc(shape: MoEShape, weights: MoEWeights, x, out, stream=None, T: int | None = None):
    """layer() without a workspace: the library's static device scratch is used
    (for callers that cannot allocate; at most 64 MiB of scratch, serialise calls)."""
    T = x.shape[0] if T is None else T
    _call(lib().ds_moe_layer_noalloc, ctypes.byref(shape.c()), ctypes.byref(weights.c()),
          x.data_ptr(), T, out.data_ptr(), _stream(stream))


def layer_resident(shape: MoEShape, weights: MoEWeights, slot, cache, experts_host, x, out, workspace,
                   debug: dict | None = None, stream=None, T: int | None = None):
    """layer() with the routed experts read through a residency view: slot [E]
    int32 (device, -1 = host), cache (device slots or None), experts_host (a
    pinned host tensor of the E packed experts)."""
    T = x.shape[0] if T is None else T
    dbg = None
    if debug is not None:
        dbg = ctypes.byref(Debug(*[_ptr(debug.get(n)) for n in
                                   ("logits", "ids", "w", "counts", "offsets", "perm")]))
    res = Residency(_ptr(slot), _ptr(cache), _ptr(experts_host))
    _call(lib().ds_moe_layer_resident, ctypes.byref(shape.c()), ctypes.byref(weights.c()), ctypes.byref(res),
          x.data_ptr(), T, out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
          dbg, _stream(stream))


def layer_path_resident(shape: MoEShape, T: int) -> int:
    rc = lib().ds_moe_layer_path_resident(ctypes.byref(shape.c()), T)
    if rc < 0:
        raise DsMoeError(rc, "invalid shape or T")
    return rc


class ExpertCache:
    """A cache of routed experts in device slots for n_layers layers (the C
    object ds_moe_cache).  experts_host: per layer a pinned host tensor of the
    E packed experts; slots: device tensor of n_slots experts (or None for a
    planning-only cache); tables: device int32 tensor [n_layers][E] (or None)."""

    def __init__(self, shape: MoEShape, experts_host, slots, n_slots: int, tables):
        self._keep = list(experts_host)
        arr = (ctypes.c_void_p * len(self._keep))(*[_host_ptr(h) for h in self._keep])
        out = ctypes.c_void_p()
        _call(lib().ds_moe_cache_create, ctypes.byref(shape.c()), len(self._keep), arr, _ptr(slots), n_slots,
              _ptr(tables), ctypes.byref(out))
        self.handle = out

    def close(self):
        if self.handle:
            lib().ds_moe_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def layer(self, layer: int, weights: MoEWeights, x, out, workspace, stream=None, T: int | None = None):
        T = x.shape[0] if T is None else T
        _call(lib().ds_moe_cache_layer, self.handle, layer, ctypes.byref(weights.c()), x.data_ptr(), T,
              out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))

    def record(self, layer: int, counts):
        """Host policy step: counts a host int32 array [E]; returns the (slot,
        expert) fills it planned."""
        import numpy as np
        c = np.ascontiguousarray(counts, np.int32)
        fills = np.empty(2 * c.size, np.int32)
        n = ctypes.c_int32()
        rc = lib().ds_moe_cache_record(self.handle, layer, c.ctypes.data, fills.ctypes.data, ctypes.byref(n))
        if rc:
            raise DsMoeError(rc, "cache record")
        return [(int(fills[2 * j]), int(fills[2 * j + 1])) for j in range(n.value)]

    def slot(self, layer: int, expert: int) -> int:
        s = ctypes.c_int32()
        rc = lib().ds_moe_cache_slot(self.handle, layer, expert, ctypes.byref(s))
        if rc:
            raise DsMoeError(rc, "cache slot")
        return s.value

    def stats(self):
        h, m, r = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        lib().ds_moe_cache_stats(self.handle, ctypes.byref(h), ctypes.byref(m), ctypes.byref(r))
        return {"hits": h.value, "misses": m.value, "resident": r.value}


def _host_ptr(t):
    """Address of a host buffer: a torch tensor or a numpy array."""
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data


def stack(shape: MoEShape, layers, x, workspace, eps: float = 1e-6, stream=None, formats=None):
    """x[T][D] fp32 residual, updated in place through len(layers) layers.
    formats: optional per-layer expert formats (DS_Q2_K / DS_Q4_K)."""
    arr = (Weights * len(layers))(*[w.c() for w in layers])
    ws = (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if formats is None:
        _call(lib().ds_moe_stack, ctypes.byref(shape.c()), arr, len(layers), x.data_ptr(),
              x.shape[0], eps, *ws, _stream(stream))
        return
    if len(formats) != len(layers):
        raise ValueError("one format per layer")
    fm = (ctypes.c_int32 * len(layers))(*formats)
    _call(lib().ds_moe_stack_mixed, ctypes.byref(shape.c()), arr, fm, len(layers), x.data_ptr(),
          x.shape[0], eps, *ws, _stream(stream))


def sync_status(stream=None):
    """Synchronise the stream and raise on a recorded device-side error."""
    _call(lib().ds_moe_sync_status, _stream(stream))


# ------------------------------------------------ one serving step around the layer


@dataclass(frozen=True)
class AttentionShape:
    """Heads, types and masks of an attention (ds_moe_attn_shape)."""
    n_head: int
    n_head_kv: int
    head_dim: int
    page_size: int
    dtype: int = DS_BF16  # or DS_F16
    scale: float = 0.0    # 0: 1 / sqrt(head_dim)
    window: int = 0       # 0: every key up to the token

    def __post_init__(self):
        c = AttnShapeC(self.n_head, self.n_head_kv, self.head_dim, self.page_size, self.dtype, self.scale, self.window)
        object.__setattr__(self, "_c", ctypes.byref(c))


class KVCache:
    """Pages of keys and values: k and v are device tensors [pages][page rows][heads][head_dim]
    of 16-bit elements and the same strides, which may be views in any order with a dense last axis
    (for instance ``kv[:, 0].transpose(1, 2)`` of pages [2][heads][rows][head_dim])."""

    def __init__(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v: [pages][page rows][heads][head_dim] of the same strides, the last axis dense")
        if k.element_size() != 2 or k.dtype != v.dtype or not (k.is_cuda and v.is_cuda):
            raise ValueError("k and v: 16-bit elements of one type on the device")
        self.k, self.v = k, v
        self._geometry = (k.size(1), k.size(2), k.size(3))
        c = KVCacheC(k.data_ptr(), v.data_ptr(), k.shape[0], k.stride(0), k.stride(1), k.stride(2))
        self._c = ctypes.byref(c)

    def _fits(self, shape: AttentionShape):
        if self._geometry != (shape.page_size, shape.n_head_kv, shape.head_dim):
            raise ValueError("the cache's pages, heads or head_dim are not the shape's")
        _half(self.k, shape, "the cache")


_types = None


def _type(t):
    """(bits, ds_dtype or None for integers) of a device tensor's elements; (0, None) on the host, or of another
    type than this binding takes."""
    global _types
    if _types is None:
        import torch
        _types = {torch.int32: (32, None), torch.int64: (64, None), torch.uint8: (8, None), torch.int16: (16, None),
                  torch.float32: (32, DS_F32), torch.bfloat16: (16, DS_BF16), torch.float16: (16, DS_F16)}
    return _types.get(t.dtype, (0, None)) if t.is_cuda else (0, None)


def _half(t, shape, name):
    # 16-bit integers are taken as the bits of the shape's type, as everywhere in this binding
    bits, kind = _type(t)
    if bits != 16 or (kind is not None and kind != shape.dtype):
        raise ValueError(f"{name}: need a device tensor of the shape's type")


_INT32, _INT64, _FLOAT32 = (32, None), (64, None), (32, DS_F32)  # _type's of arrays
_NAMES = {_INT32: "int32", _INT64: "int64", _FLOAT32: "fp32"}


def _array(t, name, kind, n=0):
    """Address of a dense device array of that type, of n elements at least."""
    if _type(t) != kind or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: need a dense device tensor of {_NAMES[kind]}, {n} elements or more")
    return t.data_ptr()


def _table(t, rows):
    if t.dim() != 2 or _type(t) != _INT32 or (t.size(1) > 1 and t.stride(1) != 1) or t.size(0) < rows:
        raise ValueError(f"block_table: need a device int32 tensor [{rows} requests][pages], rows dense")
    return t.data_ptr(), t.size(1), t.stride(0)


def page_map(context_lens, new_lens, free_pages, block_table, page_size: int, slots, positions, cu_new, seq_lens,
             n_taken, stream=None):
    """Pages and places of a step's new tokens (ds_moe_page_map): int32 device tensors, slots int64;
    block_table, slots, positions, cu_new, seq_lens and n_taken are written."""
    R, cap = context_lens.numel(), slots.numel()
    table, width, stride = _table(block_table, R)
    _call(lib().ds_moe_page_map, _array(context_lens, "context_lens", _INT32), _array(new_lens, "new_lens", _INT32, R), R,
          page_size, _array(free_pages, "free_pages", _INT32), free_pages.numel(), table, width, stride,
          _array(slots, "slots", _INT64), _array(positions, "positions", _INT32, cap), cap,
          _array(cu_new, "cu_new", _INT32, R + 1), _array(seq_lens, "seq_lens", _INT32, R), _array(n_taken, "n_taken", _INT32, 1),
          _stream(stream))


def kv_append(shape: AttentionShape, cache: KVCache, k_new, v_new, slots, stream=None):
    """Copies k_new, v_new [T][n_head_kv][head_dim] (views of any token and head stride) to their slots [T] int64."""
    cache._fits(shape)
    _half(k_new, shape, "k_new")
    strides = k_new.stride()
    if (k_new.dim() != 3 or k_new.size(1) != shape.n_head_kv or k_new.size(2) != shape.head_dim or k_new.shape != v_new.shape
            or strides != v_new.stride() or (shape.head_dim > 1 and strides[2] != 1) or k_new.dtype != v_new.dtype
            or not v_new.is_cuda):
        raise ValueError("k_new and v_new: device tensors [T][n_head_kv][head_dim] of the same strides, the last axis dense")
    T = k_new.size(0)
    _call(lib().ds_moe_kv_append, shape._c, cache._c, k_new.data_ptr(), v_new.data_ptr(), strides[0], strides[1], _array(slots, "slots", _INT64, T), T, _stream(stream))


def attention_workspace_bytes(shape: AttentionShape, n_requests: int, T: int, max_new: int) -> int:
    n = ctypes.c_size_t(0)
    _call(lib().ds_moe_attention_workspace_bytes, shape._c, n_requests, T, max_new, ctypes.byref(n))
    return n.value


def _rows(t, shape, name):
    s0, s1, s2 = t.stride() if t.dim() == 3 else (0, 0, 0)
    if (s1 == 0 or t.size(1) != shape.n_head or t.size(2) != shape.head_dim
            or (shape.head_dim > 1 and s2 != 1) or (shape.n_head > 1 and s1 != shape.head_dim)):
        raise ValueError(f"{name}: need a device tensor [T][n_head][head_dim] with dense heads")
    _half(t, shape, name)
    return t.data_ptr(), s0


def paged_attention(shape: AttentionShape, cache: KVCache, block_table, q, cu_new, seq_lens, max_new: int, out, workspace,
                    lse=None, stream=None):
    """out[T][n_head][head_dim] = attention of the new tokens q over the cache's pages (ds_moe_paged_attention);
    lse: optional fp32 [T][n_head].  block_table, cu_new and seq_lens as page_map writes them."""
    cache._fits(shape)
    R, T = seq_lens.numel(), q.size(0)
    qp, qs = _rows(q, shape, "q")
    op, os_ = _rows(out, shape, "out")
    table, width, stride = _table(block_table, R)
    if out.size(0) < T:
        raise ValueError("out has too few rows")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace: need a dense device tensor")
    room = workspace.numel() * workspace.element_size()
    _call(lib().ds_moe_paged_attention, shape._c, cache._c, table, width, stride, qp, qs, T, _array(cu_new, "cu_new", _INT32, R + 1),
          _array(seq_lens, "seq_lens", _INT32), R, max_new, op, os_,
          None if lse is None else _array(lse, "lse", _FLOAT32, T * shape.n_head), workspace.data_ptr(), room,
          _stream(stream))


def attention_path(shape: AttentionShape, cache: KVCache, q, max_new: int) -> int:
    """Which kernels paged_attention runs (an ATTN_* value) with a table of one column or more."""
    stride = q.stride(0) if q.size(0) > 1 else shape.n_head * shape.head_dim  # (a lone token's is not used)
    rc = lib().ds_moe_attention_path(shape._c, cache._c, q.data_ptr(), stride, max_new)
    if rc < 0:
        raise DsMoeError(rc, "shape, cache or max_new rejected")
    return rc


def verify_drafts(target, draft, tokens, cu_new, u_accept, u_sample, out_tokens, n_accepted, stream=None):
    """Checks drafted tokens against target [T][vocab] (fp32 or bf16 probabilities) from given random numbers
    (ds_moe_verify_drafts).  draft: the drafter's probabilities, rows as target's, or None; out_tokens
    [requests][max_new] and n_accepted [requests] int32 are written."""
    strides = target.stride()
    kind = _type(target)[1]
    if target.dim() != 2 or kind not in (DS_F32, DS_BF16) or (target.size(1) > 1 and strides[1] != 1):
        raise ValueError("target: need a device tensor [T][vocab] of fp32 or bf16, rows dense")
    if draft is not None and (draft.shape != target.shape or draft.dtype != target.dtype or not draft.is_cuda or
                              (draft.size(1) > 1 and draft.stride(1) != 1)):
        raise ValueError("draft: need a tensor like target")
    R, T, V = n_accepted.numel(), target.size(0), target.size(1)
    if out_tokens.dim() != 2 or out_tokens.size(0) != R:
        raise ValueError("out_tokens: need [requests][max_new]")
    _call(lib().ds_moe_verify_drafts, target.data_ptr(), strides[0], _ptr(draft), 0 if draft is None else draft.stride(0),
          kind, T, V, _array(tokens, "tokens", _INT32, T),
          _array(cu_new, "cu_new", _INT32, R + 1), R, out_tokens.size(1), _array(u_accept, "u_accept", _FLOAT32, T),
          _array(u_sample, "u_sample", _FLOAT32, R), _array(out_tokens, "out_tokens", _INT32), _array(n_accepted, "n_accepted", _INT32),
          _stream(stream))
