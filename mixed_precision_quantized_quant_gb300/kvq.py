"""Thin ctypes binding of libkvq.so (include/kvq.h).

Argument marshalling only: every step of quantization and attention runs in
the library's CUDA kernels.  PyTorch provides the device memory and streams.
The functions keep the C names; ``KVQCache`` bundles them for convenience.
There is no fallback: if the library is not built, loading it raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
# KVQ_DEBUG_LIB=1 selects the debug build (device-side range checks of every
# computed access, reported through the error word)
LIB_PATH = os.path.join(_HERE, "libkvq_debug.so" if os.environ.get("KVQ_DEBUG_LIB") == "1" else "libkvq.so")

STATUS = {
    0: "KVQ_OK", 1: "KVQ_ERR_ARG", 2: "KVQ_ERR_BITS", 3: "KVQ_ERR_ALIGN", 4: "KVQ_ERR_CAPACITY",
    5: "KVQ_ERR_CUDA", 6: "KVQ_ERR_STATE", 7: "KVQ_ERR_UNSUPPORTED",
}

EXPORTS = (
    "kvq_cache_bytes", "kvq_create", "kvq_append", "kvq_decode_attn", "kvq_decode_step",
    "kvq_layer_view_get", "kvq_equivalent_bits", "kvq_decode_bytes", "kvq_device_error",
    "kvq_destroy", "kvq_status_string", "kvq_decode_attn_noalloc", "kvq_chunk_attn",
    "kvq_selftest_bounded_wait", "kvq_chunk_workspace_bytes", "kvq_state_bytes", "kvq_state_save",
    "kvq_state_restore",
    "kvq_paged_bytes", "kvq_paged_create", "kvq_paged_append", "kvq_paged_decode_attn", "kvq_paged_workspace_bytes",
    "kvq_paged_read", "kvq_paged_view_get", "kvq_paged_device_error", "kvq_paged_destroy",
)


class KVQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


KEY_PER_CHANNEL, KEY_PER_TOKEN = 0, 1


class LayerCfg(ctypes.Structure):
    _fields_ = [("k_bits", ctypes.c_uint8), ("v_bits", ctypes.c_uint8), ("key_mode", ctypes.c_uint8),
                ("rpc_percent", ctypes.c_uint8), ("residual", ctypes.c_int32)]


class Config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("layers", ctypes.POINTER(LayerCfg))]


class LayerView(ctypes.Structure):
    _fields_ = [("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32), ("residual", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k_words", ctypes.c_int32), ("v_words", ctypes.c_int32), ("key_mode", ctypes.c_int32),
                ("record_bytes", ctypes.c_int64), ("unit_record_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64), ("tokens", ctypes.c_int64),
                ("quantized_tokens", ctypes.c_int64), ("residual_tokens", ctypes.c_int64),
                ("records", ctypes.c_void_p), ("residual_k", ctypes.c_void_p),
                ("residual_v", ctypes.c_void_p), ("window_bound", ctypes.c_int32),
                ("rpc_percent", ctypes.c_int32)]


KVQ_FP16, KVQ_BF16 = 0, 1
_FLT_MIN = 2.0 ** -126


class PagedLayerCfg(ctypes.Structure):
    _fields_ = [("k_bits", ctypes.c_uint8), ("v_bits", ctypes.c_uint8)]


class PagedConfig(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("layers", ctypes.POINTER(PagedLayerCfg))]


class PagedView(ctypes.Structure):
    _fields_ = [("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("tile_bytes", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("pages", ctypes.c_void_p)]


class PagedBatchArgs(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("seq_lens", ctypes.c_void_p),
                ("cu_tokens", ctypes.c_void_p), ("num_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class RotationArgs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libkvq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} is missing: build it with mixed_precision_quantized_quant_gb300.build.build()")
    L = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.kvq_cache_bytes.argtypes = [ctypes.POINTER(Config)]
    L.kvq_cache_bytes.restype = ctypes.c_size_t
    L.kvq_create.argtypes = [ctypes.POINTER(Config), vp, ctypes.c_size_t, ctypes.POINTER(vp)]
    L.kvq_create.restype = ctypes.c_int
    L.kvq_append.argtypes = [vp, ctypes.c_int, vp, vp, ctypes.c_int, vp]
    L.kvq_append.restype = ctypes.c_int
    L.kvq_decode_attn.argtypes = [vp, ctypes.c_int, vp, vp, vp]
    L.kvq_decode_attn.restype = ctypes.c_int
    L.kvq_decode_attn_noalloc.argtypes = [vp, ctypes.c_int, vp, vp, vp]
    L.kvq_decode_attn_noalloc.restype = ctypes.c_int
    L.kvq_chunk_attn.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, ctypes.c_size_t, vp]
    L.kvq_chunk_attn.restype = ctypes.c_int
    L.kvq_chunk_workspace_bytes.argtypes = [vp]
    L.kvq_chunk_workspace_bytes.restype = ctypes.c_size_t
    L.kvq_decode_step.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                  ctypes.POINTER(vp), vp]
    L.kvq_decode_step.restype = ctypes.c_int
    L.kvq_layer_view_get.argtypes = [vp, ctypes.c_int, ctypes.POINTER(LayerView)]
    L.kvq_layer_view_get.restype = ctypes.c_int
    L.kvq_equivalent_bits.argtypes = [vp]
    L.kvq_equivalent_bits.restype = ctypes.c_double
    L.kvq_decode_bytes.argtypes = [vp, ctypes.c_int]
    L.kvq_decode_bytes.restype = i64
    L.kvq_device_error.argtypes = [vp, ctypes.POINTER(i32), vp]
    L.kvq_device_error.restype = ctypes.c_int
    L.kvq_selftest_bounded_wait.argtypes = [vp, vp]
    L.kvq_selftest_bounded_wait.restype = ctypes.c_int
    L.kvq_state_bytes.argtypes = [vp]
    L.kvq_state_bytes.restype = ctypes.c_size_t
    L.kvq_state_save.argtypes = [vp, vp, vp]
    L.kvq_state_save.restype = ctypes.c_int
    L.kvq_state_restore.argtypes = [vp, vp, vp]
    L.kvq_state_restore.restype = ctypes.c_int
    L.kvq_destroy.argtypes = [vp]
    L.kvq_destroy.restype = ctypes.c_int
    L.kvq_status_string.argtypes = [ctypes.c_int]
    L.kvq_status_string.restype = ctypes.c_char_p
    batch, rows = ctypes.POINTER(PagedBatchArgs), ctypes.POINTER(Rows)
    L.kvq_paged_bytes.argtypes = [ctypes.POINTER(PagedConfig)]
    L.kvq_paged_bytes.restype = ctypes.c_size_t
    L.kvq_paged_create.argtypes = [ctypes.POINTER(PagedConfig), vp, ctypes.c_size_t, ctypes.POINTER(vp)]
    L.kvq_paged_create.restype = ctypes.c_int
    L.kvq_paged_append.argtypes = [vp, ctypes.c_int, batch, rows, rows, rows, rows, ctypes.POINTER(RotationArgs),
                                   ctypes.c_int, vp]
    L.kvq_paged_append.restype = ctypes.c_int
    L.kvq_paged_decode_attn.argtypes = [vp, ctypes.c_int, batch, rows, vp, vp, ctypes.c_float, ctypes.c_int, vp,
                                        ctypes.c_size_t, vp]
    L.kvq_paged_decode_attn.restype = ctypes.c_int
    L.kvq_paged_workspace_bytes.argtypes = [vp, ctypes.c_int]
    L.kvq_paged_workspace_bytes.restype = ctypes.c_size_t
    L.kvq_paged_read.argtypes = [vp, ctypes.c_int, batch, rows, rows, ctypes.c_int, vp]
    L.kvq_paged_read.restype = ctypes.c_int
    L.kvq_paged_view_get.argtypes = [vp, ctypes.c_int, ctypes.POINTER(PagedView)]
    L.kvq_paged_view_get.restype = ctypes.c_int
    L.kvq_paged_device_error.argtypes = [vp, ctypes.POINTER(i32), vp]
    L.kvq_paged_device_error.restype = ctypes.c_int
    L.kvq_paged_destroy.argtypes = [vp]
    L.kvq_paged_destroy.restype = ctypes.c_int
    _lib = L
    return L


def _check(st: int, where: str) -> None:
    if st != 0:
        raise KVQError(st, where)


def make_config(layers: Sequence[Tuple[int, ...]], batch: int, num_q_heads: int, num_kv_heads: int,
                head_dim: int, group_size: int, max_tokens: int):
    """layers: (k_bits, v_bits, residual[, key_mode[, rpc_percent]]) per layer."""
    arr = (LayerCfg * len(layers))()
    for i, spec in enumerate(layers):
        kb, vb, r = spec[:3]
        km = spec[3] if len(spec) > 3 else KEY_PER_CHANNEL
        rpc = spec[4] if len(spec) > 4 else 0
        arr[i].k_bits, arr[i].v_bits, arr[i].key_mode, arr[i].rpc_percent, arr[i].residual = kb, vb, km, rpc, r
    cfg = Config(len(layers), batch, num_q_heads, num_kv_heads, head_dim, group_size, max_tokens,
                 ctypes.cast(arr, ctypes.POINTER(LayerCfg)))
    cfg._keep = arr  # keep the layer array alive with the struct
    return cfg


# ---------------------------------------------------------------- C names

def kvq_cache_bytes(cfg: Config) -> int:
    return int(load().kvq_cache_bytes(ctypes.byref(cfg)))


def kvq_create(cfg: Config, dev_buf: int, nbytes: int) -> int:
    h = ctypes.c_void_p()
    _check(load().kvq_create(ctypes.byref(cfg), ctypes.c_void_p(dev_buf), nbytes, ctypes.byref(h)), "kvq_create")
    return h.value


def kvq_append(h: int, layer: int, K: int, V: int, n_tokens: int, stream: int) -> None:
    _check(load().kvq_append(h, layer, K, V, n_tokens, stream), "kvq_append")


def kvq_decode_attn(h: int, layer: int, q: int, out: int, stream: int) -> None:
    _check(load().kvq_decode_attn(h, layer, q, out, stream), "kvq_decode_attn")


def kvq_decode_attn_noalloc(h: int, layer: int, q: int, out: int, stream: int) -> None:
    """kvq_decode_attn with the library's static device scratch: for callers
    that may not allocate device memory (see include/kvq.h)."""
    _check(load().kvq_decode_attn_noalloc(h, layer, q, out, stream), "kvq_decode_attn_noalloc")


def kvq_chunk_attn(h: int, layer: int, q: int, n_queries: int, out: int, workspace: int, workspace_bytes: int,
                   stream: int) -> None:
    _check(load().kvq_chunk_attn(h, layer, q, n_queries, out, workspace, workspace_bytes, stream), "kvq_chunk_attn")


def kvq_chunk_workspace_bytes(h: int) -> int:
    return int(load().kvq_chunk_workspace_bytes(h))


def kvq_decode_step(h: int, K: Sequence[int], V: Sequence[int], q: Sequence[int], out: Sequence[int],
                    stream: int) -> None:
    n = len(K)
    arr = [(ctypes.c_void_p * n)(*x) for x in (K, V, q, out)]
    _check(load().kvq_decode_step(h, *arr, stream), "kvq_decode_step")


def kvq_layer_view_get(h: int, layer: int) -> dict:
    v = LayerView()
    _check(load().kvq_layer_view_get(h, layer, ctypes.byref(v)), "kvq_layer_view_get")
    return {name: getattr(v, name) for name, _ in LayerView._fields_}


def kvq_equivalent_bits(h: int) -> float:
    return float(load().kvq_equivalent_bits(h))


def kvq_decode_bytes(h: int, layer: int) -> int:
    return int(load().kvq_decode_bytes(h, layer))


def kvq_device_error(h: int, stream: int) -> int:
    code = ctypes.c_int32(0)
    _check(load().kvq_device_error(h, ctypes.byref(code), stream), "kvq_device_error")
    return code.value


def kvq_selftest_bounded_wait(h: int, stream: int) -> None:
    _check(load().kvq_selftest_bounded_wait(h, stream), "kvq_selftest_bounded_wait")


def kvq_state_bytes(h: int) -> int:
    return int(load().kvq_state_bytes(h))


def kvq_state_save(h: int, dst: int, stream: int) -> None:
    _check(load().kvq_state_save(h, dst, stream), "kvq_state_save")


def kvq_state_restore(h: int, src: int, stream: int) -> None:
    _check(load().kvq_state_restore(h, src, stream), "kvq_state_restore")


def kvq_destroy(h: int) -> None:
    _check(load().kvq_destroy(h), "kvq_destroy")


def make_paged_config(layers: Sequence[Tuple[int, int]], num_q_heads: int, num_kv_heads: int, head_dim: int,
                      page_size: int, num_pages: int, dtype: int = KVQ_FP16):
    """layers: (k_bits, v_bits) per layer; dtype: KVQ_FP16 or KVQ_BF16."""
    sizes = (num_q_heads, num_kv_heads, head_dim, page_size, num_pages, dtype)
    if any(not -2 ** 31 <= x < 2 ** 31 for x in sizes) or any(not 0 <= b < 256 for x in layers for b in x):
        raise ValueError("a size that 32 bits, or a width that 8 bits do not hold")  # C types would cut it
    arr = (PagedLayerCfg * len(layers))()
    for i, (kb, vb) in enumerate(layers):
        arr[i].k_bits, arr[i].v_bits = kb, vb
    cfg = PagedConfig(len(layers), num_q_heads, num_kv_heads, head_dim, page_size, num_pages, dtype,
                      ctypes.cast(arr, ctypes.POINTER(PagedLayerCfg)))
    cfg._keep = arr
    return cfg


def kvq_paged_bytes(cfg: PagedConfig) -> int:
    return int(load().kvq_paged_bytes(ctypes.byref(cfg)))


def kvq_paged_create(cfg: PagedConfig, dev_buf: int, nbytes: int) -> int:
    h = ctypes.c_void_p()
    _check(load().kvq_paged_create(ctypes.byref(cfg), ctypes.c_void_p(dev_buf), nbytes, ctypes.byref(h)),
           "kvq_paged_create")
    return h.value


def kvq_paged_append(h: int, layer: int, batch: PagedBatchArgs, K: Rows, V: Rows, q: Optional[Rows],
                     q_out: Optional[Rows], rotation: Optional[RotationArgs], n_tokens: int, stream: int) -> None:
    _check(load().kvq_paged_append(h, layer, batch, K, V, q, q_out, rotation, n_tokens, stream), "kvq_paged_append")


def kvq_paged_decode_attn(h: int, layer: int, batch: PagedBatchArgs, q: Rows, out: int, lse: Optional[int],
                          scale: float, window: int, workspace: int, workspace_bytes: int, stream: int) -> None:
    _check(load().kvq_paged_decode_attn(h, layer, batch, q, out, lse, scale, window, workspace, workspace_bytes,
                                        stream), "kvq_paged_decode_attn")


def kvq_paged_workspace_bytes(h: int, num_seqs: int) -> int:
    return int(load().kvq_paged_workspace_bytes(h, num_seqs))


def kvq_paged_read(h: int, layer: int, batch: PagedBatchArgs, K: Optional[Rows], V: Optional[Rows], n_tokens: int,
                   stream: int) -> None:
    _check(load().kvq_paged_read(h, layer, batch, K, V, n_tokens, stream), "kvq_paged_read")


def kvq_paged_view_get(h: int, layer: int) -> dict:
    v = PagedView()
    _check(load().kvq_paged_view_get(h, layer, ctypes.byref(v)), "kvq_paged_view_get")
    return {name: getattr(v, name) for name, _ in PagedView._fields_}


def kvq_paged_device_error(h: int, stream: int) -> int:
    code = ctypes.c_int32(0)
    _check(load().kvq_paged_device_error(h, ctypes.byref(code), stream), "kvq_paged_device_error")
    return code.value


def kvq_paged_destroy(h: int) -> None:
    _check(load().kvq_paged_destroy(h), "kvq_paged_destroy")


def kvq_status_string(s: int) -> str:
    return load().kvq_status_string(s).decode()


# ---------------------------------------------------------------- convenience

def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _dev_ptr(t, name: str, dtype, shape) -> int:
    import torch
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return int(t.data_ptr())


class KVQCache:
    """A layer-wise mixed-precision KV cache living in one torch-allocated
    device buffer."""

    def __init__(self, layers: Sequence[Tuple[int, int, int]], batch: int, num_q_heads: int,
                 num_kv_heads: int, head_dim: int, group_size: int, max_tokens: int, device="cuda"):
        import torch
        self.layers = [tuple(x) for x in layers]
        self.B, self.Hq, self.Hkv, self.D, self.G = batch, num_q_heads, num_kv_heads, head_dim, group_size
        self.max_tokens = max_tokens
        self.cfg = make_config(self.layers, batch, num_q_heads, num_kv_heads, head_dim, group_size, max_tokens)
        self.nbytes = kvq_cache_bytes(self.cfg)
        if self.nbytes == 0:
            raise KVQError(1, "kvq_cache_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.h = kvq_create(self.cfg, int(self.buf.data_ptr()), self.nbytes)

    def append(self, layer: int, K, V, stream=None) -> None:
        import torch
        n = K.shape[2]
        shp = (self.B, self.Hkv, n, self.D)
        kvq_append(self.h, layer, _dev_ptr(K, "K", torch.float16, shp), _dev_ptr(V, "V", torch.float16, shp),
                   n, _stream_ptr(stream))

    def decode_attn(self, layer: int, q, out=None, stream=None):
        import torch
        if out is None:
            out = torch.empty((self.B, self.Hq, self.D), dtype=torch.float32, device=q.device)
        kvq_decode_attn(self.h, layer, _dev_ptr(q, "q", torch.float16, (self.B, self.Hq, self.D)),
                        _dev_ptr(out, "out", torch.float32, (self.B, self.Hq, self.D)), _stream_ptr(stream))
        return out

    def chunk_attn(self, layer: int, q, out=None, stream=None):
        """Causal attention of the queries of the newest q.shape[2] tokens:
        q fp16 [B, Hq, n, d] -> fp32 [B, Hq, n, d]."""
        import torch
        n = int(q.shape[2])
        shp = (self.B, self.Hq, n, self.D)
        if out is None:
            out = torch.empty(shp, dtype=torch.float32, device=q.device)
        if getattr(self, "_chunk_ws", None) is None:  # allocated on first use, kept with the cache
            self._chunk_ws = torch.empty(kvq_chunk_workspace_bytes(self.h), dtype=torch.uint8, device=self.buf.device)
        kvq_chunk_attn(self.h, layer, _dev_ptr(q, "q", torch.float16, shp), n,
                       _dev_ptr(out, "out", torch.float32, shp), int(self._chunk_ws.data_ptr()),
                       self._chunk_ws.numel(), _stream_ptr(stream))
        return out

    def decode_step(self, K: List, V: List, q: List, out: List, stream=None) -> None:
        import torch
        kv = (self.B, self.Hkv, 1, self.D)
        qs = (self.B, self.Hq, self.D)
        kvq_decode_step(self.h,
                        [_dev_ptr(x, "K", torch.float16, kv) for x in K],
                        [_dev_ptr(x, "V", torch.float16, kv) for x in V],
                        [_dev_ptr(x, "q", torch.float16, qs) for x in q],
                        [_dev_ptr(x, "out", torch.float32, qs) for x in out],
                        _stream_ptr(stream))

    def view(self, layer: int) -> dict:
        return kvq_layer_view_get(self.h, layer)

    def equivalent_bits(self) -> float:
        return kvq_equivalent_bits(self.h)

    def decode_bytes(self, layer: int) -> int:
        return kvq_decode_bytes(self.h, layer)

    def device_error(self, stream=None) -> int:
        return kvq_device_error(self.h, _stream_ptr(stream))

    def save_state(self, snapshot=None, stream=None):
        """Snapshot of the streaming state (token counters and FP16 windows of
        every layer) into a uint8 device tensor of kvq_state_bytes bytes,
        allocated if not given; returns it."""
        import torch
        n = kvq_state_bytes(self.h)
        if snapshot is None:
            snapshot = torch.empty(n, dtype=torch.uint8, device=self.buf.device)
        kvq_state_save(self.h, _dev_ptr(snapshot, "snapshot", torch.uint8, (n,)), _stream_ptr(stream))
        return snapshot

    def restore_state(self, snapshot, stream=None) -> None:
        import torch
        n = kvq_state_bytes(self.h)
        kvq_state_restore(self.h, _dev_ptr(snapshot, "snapshot", torch.uint8, (n,)), _stream_ptr(stream))

    def close(self) -> None:
        if getattr(self, "h", None):
            kvq_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _device_tensor(t, name: str, dtype, device, ndim: int) -> None:
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")


class PagedBatch:
    """The sequences that calls of a ``KVQPagedCache`` work on: int32 CUDA
    tensors, read on the device at every call (one batch serves every layer,
    and a captured step follows what is copied into them later).

    page_table [S, max_pages]: page of every page_size positions;
    seq_lens [S]: tokens of each sequence, the new ones included;
    cu_tokens [S + 1] or None: rows cu_tokens[s] .. cu_tokens[s+1] - 1 of an
    append's or a read's tensors are the newest of sequence s (None: row s)."""

    def __init__(self, page_table, seq_lens, cu_tokens=None):
        import torch
        dev = page_table.device
        if dev.type != "cuda":
            raise ValueError("page_table must be a CUDA tensor")
        _device_tensor(page_table, "page_table", torch.int32, dev, 2)
        _device_tensor(seq_lens, "seq_lens", torch.int32, dev, 1)
        S, width = page_table.shape
        if S < 1 or width < 1:
            raise ValueError(f"page_table has shape {tuple(page_table.shape)}: at least one sequence and one page")
        if width > 1 and page_table.stride(1) != 1:
            raise ValueError("page_table rows must be contiguous")
        stride = page_table.stride(0) if S > 1 else width
        if stride < width:
            raise ValueError("page_table rows must not overlap")
        if tuple(seq_lens.shape) != (S,) or not seq_lens.is_contiguous():
            raise ValueError(f"seq_lens must be contiguous of shape {(S,)}")
        if cu_tokens is not None:
            _device_tensor(cu_tokens, "cu_tokens", torch.int32, dev, 1)
            if tuple(cu_tokens.shape) != (S + 1,) or not cu_tokens.is_contiguous():
                raise ValueError(f"cu_tokens must be contiguous of shape {(S + 1,)}")
        self.device, self.num_seqs = dev, S
        self._keep = (page_table, seq_lens, cu_tokens)
        self.args = PagedBatchArgs(page_table.data_ptr(), stride, seq_lens.data_ptr(),
                                   None if cu_tokens is None else cu_tokens.data_ptr(), S, width)


class Rotation:
    """The position rotation of an append: table fp32 [rows, dim] on the GPU,
    dim / 2 cosines then dim / 2 sines of each position's angles (see
    ``rotation_table``); positions int32 [n_tokens] or None (each row's place
    in its sequence); interleaved pairs channels (2i, 2i+1) instead of
    (i, i + dim/2)."""

    def __init__(self, table, interleaved: bool = False, positions=None):
        import torch
        if table.device.type != "cuda":
            raise ValueError("table must be a CUDA tensor")
        _device_tensor(table, "table", torch.float32, table.device, 2)
        rows, dim = table.shape
        if not table.is_contiguous() or rows < 1:
            raise ValueError("table must be contiguous with at least one row")
        if dim < 16 or dim % 16:
            raise ValueError(f"table has {dim} columns: a multiple of 16 is needed")
        self.positions = None
        if positions is not None:
            _device_tensor(positions, "positions", torch.int32, table.device, 1)
            if not positions.is_contiguous():
                raise ValueError("positions must be contiguous")
            self.positions = positions
        self.table, self.dim, self.device = table, dim, table.device
        self.args = RotationArgs(table.data_ptr(), None if positions is None else positions.data_ptr(), rows, dim,
                                 int(bool(interleaved)))


def rotation_table(rows: int, dim: int, base: float = 10000.0, device="cuda"):
    """Cosines and sines of p * base^(-2i/dim) for positions p < rows, in the
    form ``Rotation`` takes; the angles are formed in 64 bits (far positions
    lose theirs in 32)."""
    import torch
    inv = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    ang = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


class KVQPagedCache:
    """A paged cache of ``num_pages`` pages of ``page_size`` tokens per layer,
    each layer at its own (k_bits, v_bits): (16, 16) keeps rows in ``dtype``,
    smaller pairs from {2, 4, 8} quantize them per token (see include/kvq.h).
    ``buffer``: uint8 CUDA tensor of ``nbytes`` bytes to use, else one is made.
    Which pages belong to which sequence is the caller's: a call takes a
    ``PagedBatch``.  Tensors of rows are [n, heads, head_dim] with contiguous
    head_dim, such as slices of a projection's output."""

    def __init__(self, layers: Sequence[Tuple[int, int]], num_q_heads: int, num_kv_heads: int, head_dim: int,
                 page_size: int, num_pages: int, dtype=None, device="cuda", buffer=None):
        import torch
        self.h = None
        dtype = torch.float16 if dtype is None else dtype
        if dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"dtype must be torch.float16 or torch.bfloat16, got {dtype}")
        self.layers = [tuple(x) for x in layers]
        self.Hq, self.Hkv, self.D, self.P = num_q_heads, num_kv_heads, head_dim, page_size
        self.num_pages, self.dtype = num_pages, dtype
        self.cfg = make_paged_config(self.layers, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                                     KVQ_FP16 if dtype == torch.float16 else KVQ_BF16)
        self.nbytes = kvq_paged_bytes(self.cfg)
        if self.nbytes == 0:
            raise KVQError(1, "kvq_paged_bytes")
        if buffer is None:
            buffer = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        elif not buffer.is_cuda or buffer.dtype != torch.uint8 or buffer.dim() != 1 or not buffer.is_contiguous():
            raise ValueError("buffer must be a contiguous one-dimensional uint8 CUDA tensor")
        self.buf, self.device = buffer, buffer.device
        with torch.cuda.device(self.device):
            # the library writes its own bytes with the device idle behind it
            torch.cuda.current_stream().synchronize()
            self.h = kvq_paged_create(self.cfg, int(buffer.data_ptr()), buffer.numel())
        self._ws = {}  # num_seqs -> workspace bytes
        # a decode step makes two of these calls for every layer, so what a
        # call looks up is kept here
        lib = load()
        self._c_append, self._c_attn, self._c_read = lib.kvq_paged_append, lib.kvq_paged_decode_attn, lib.kvq_paged_read
        self._empty, self._f32, self._u8 = torch.empty, torch.float32, torch.uint8
        self._raw_stream, self._index = torch._C._cuda_getCurrentRawStream, self.device.index
        self._current_device, self._device_guard = torch._C._cuda_getDevice, torch.cuda.device
        self._stream_guard = torch.cuda.stream

    def _rows(self, t, name: str, n: int, heads: int) -> Rows:
        if t.dtype is self.dtype and t.shape == (n, heads, self.D) and t.device == self.device:
            a, b, c = t.stride()
            if c == 1:
                return Rows(t.data_ptr(), a, b)
            raise ValueError(f"{name}'s last dimension must be contiguous")
        if tuple(t.shape) != (n, heads, self.D):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n, heads, self.D)}")
        raise ValueError(f"{name} must be {self.dtype} on {self.device}, got {t.dtype} on {t.device}")

    def _out_rows(self, t, name: str, n: int, heads: int) -> Rows:
        """Rows to write, none of which may share a place with another."""
        r, d = self._rows(t, name, n, heads), self.D
        a, b = r.token_stride, r.head_stride
        if (n > 1 and a < d) or (heads > 1 and b < d) or \
                (n > 1 and heads > 1 and a < (heads - 1) * b + d and b < (n - 1) * a + d):
            raise ValueError(f"{name}'s rows overlap one another")
        return r

    def _new(self, stream, shape, dtype):
        """An output or scratch tensor that the allocator ties to the call's stream."""
        if stream is None:
            return self._empty(shape, dtype=dtype, device=self.device)
        with self._stream_guard(stream):
            return self._empty(shape, dtype=dtype, device=self.device)

    def _batch(self, batch: PagedBatch) -> PagedBatchArgs:
        if batch.device != self.device:
            raise ValueError(f"batch must be on {self.device}, got {batch.device}")
        return batch.args

    def _counts(self, layer: int, n: int, where: str) -> None:
        """Refuses what a C int would cut to another number."""
        if not 0 <= layer < len(self.layers) or not 0 <= n < 2 ** 31:
            raise KVQError(1, where)

    def _stream(self, stream) -> int:
        return self._raw_stream(self._index) if stream is None else stream.cuda_stream

    def _on_device(self, fn, *args) -> int:
        with self._device_guard(self.device):
            return fn(*args)

    def append(self, layer: int, batch: PagedBatch, K, V, q=None, rotation: Optional[Rotation] = None, q_out=None,
               stream=None):
        """Appends the newest rows of every sequence: K, V [n, Hkv, d]; returns
        q [n, Hq, d] turned by ``rotation`` (into ``q_out``, which may be q), or
        None without q.  Rows of q_out that belong to no sequence are not
        written."""
        n = K.shape[0]
        self._counts(layer, n, "kvq_paged_append")
        k, v = self._rows(K, "K", n, self.Hkv), self._rows(V, "V", n, self.Hkv)
        b = self._batch(batch)
        if b.cu_tokens is None and n != batch.num_seqs:
            raise ValueError(f"K has {n} rows, expected one for each of {batch.num_seqs} sequences")
        r = qr = qo = None
        if rotation is not None:
            if rotation.device != self.device or rotation.dim > self.D:
                raise ValueError(f"rotation must be on {self.device} and turn at most {self.D} channels")
            if rotation.positions is not None and rotation.positions.numel() < n:
                raise ValueError(f"rotation has {rotation.positions.numel()} positions, expected {n}")
            r = rotation.args
        if q is not None:
            qr = self._rows(q, "q", n, self.Hq)
            if q_out is None:
                q_out = self._new(stream, (n, self.Hq, self.D), self.dtype)
            qo = self._out_rows(q_out, "q_out", n, self.Hq)
        elif q_out is not None:
            raise ValueError("q_out without q")
        args = self.h, layer, b, k, v, qr, qo, r, n, self._stream(stream)
        st = self._c_append(*args) if self._current_device() == self._index else self._on_device(self._c_append, *args)
        if st:
            raise KVQError(st, "kvq_paged_append")
        return q_out

    def decode_attn(self, layer: int, batch: PagedBatch, q, out=None, scale: float = 0.0, window: int = 0,
                    return_lse: bool = False, stream=None):
        """Attention of one query per sequence over its newest ``window``
        tokens (0: all): q [S, Hq, d] -> [S, Hq, d] in the cache's dtype, and
        with return_lse (out, fp32 [S, Hq] log-sum-exp of the scaled scores)."""
        S = batch.num_seqs
        self._counts(layer, window, "kvq_paged_decode_attn")
        b = self._batch(batch)
        qr = self._rows(q, "q", S, self.Hq)
        if out is None:
            out = self._new(stream, (S, self.Hq, self.D), self.dtype)
        elif out.dtype != self.dtype or out.device != self.device or tuple(out.shape) != (S, self.Hq, self.D) or \
                not out.is_contiguous():
            raise ValueError(f"out must be contiguous {self.dtype} of shape {(S, self.Hq, self.D)} on {self.device}")
        lse = self._new(stream, (S, self.Hq), self._f32) if return_lse else None
        if scale and -_FLT_MIN < scale < _FLT_MIN:  # as a C float it could be 0, which means another scale
            raise ValueError(f"scale must be 0 or at least {_FLT_MIN} in magnitude, got {scale}")
        nws = self._ws.get(S)
        if nws is None:
            nws = self._ws[S] = kvq_paged_workspace_bytes(self.h, S)
        # every call has a workspace of its own, so that calls on several
        # streams, or of several captured graphs, never share one
        ws = self._new(stream, nws, self._u8)
        args = (self.h, layer, b, qr, out.data_ptr(), lse.data_ptr() if return_lse else None, scale, window,
                ws.data_ptr(), nws, self._stream(stream))
        st = self._c_attn(*args) if self._current_device() == self._index else self._on_device(self._c_attn, *args)
        if st:
            raise KVQError(st, "kvq_paged_decode_attn")
        return (out, lse) if return_lse else out

    def read(self, layer: int, batch: PagedBatch, n: int, K=None, V=None, stream=None):
        """The newest rows of every sequence as the cache holds them: (K, V),
        [n, Hkv, d] in the cache's dtype; rows that belong to no sequence are
        not written."""
        self._counts(layer, n, "kvq_paged_read")
        b = self._batch(batch)
        if b.cu_tokens is None and n != batch.num_seqs:
            raise ValueError(f"n is {n}, expected one row for each of {batch.num_seqs} sequences")
        if K is None:
            K = self._new(stream, (n, self.Hkv, self.D), self.dtype)
        if V is None:
            V = self._new(stream, (n, self.Hkv, self.D), self.dtype)
        k, v = self._out_rows(K, "K", n, self.Hkv), self._out_rows(V, "V", n, self.Hkv)
        args = self.h, layer, b, k, v, n, self._stream(stream)
        st = self._c_read(*args) if self._current_device() == self._index else self._on_device(self._c_read, *args)
        if st:
            raise KVQError(st, "kvq_paged_read")
        return K, V

    def view(self, layer: int) -> dict:
        self._counts(layer, 0, "kvq_paged_view_get")
        return kvq_paged_view_get(self.h, layer)

    def device_error(self, stream=None) -> int:
        with self._device_guard(self.device):
            return kvq_paged_device_error(self.h, _stream_ptr(stream))

    def close(self) -> None:
        if getattr(self, "h", None):
            kvq_paged_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
