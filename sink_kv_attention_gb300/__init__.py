"""Python binding of libsinkkv (sink + window KV attention with RoPE/YaRN on GB300).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels, reached through the C ABI declared in ``include/sinkkv.h``.  PyTorch
tensors supply device memory and the current CUDA stream.  There is no CPU
fallback: if ``libsinkkv.so`` is missing or fails to load, importing the binding's
functions raises.

C entry point          Python
sk_rope_table_*        RopeTable (+ rope_table_fill_host)
sk_rope_dynamic_*      DynamicRope (+ dynamic_factor)
sk_rope_apply          rope_apply
sk_kv_append           kv_append
sk_decode_attention    decode_attention (+ decode_workspace_bytes, decode_attention_noalloc)
sk_decode_step         decode_step (+ decode_step_workspace_bytes)
sk_prefill_attention   prefill_attention
sk_kv_rerotate         kv_rerotate
sk_kv_shift_recent     kv_shift_recent
sk_paged_*             PagedLayer, paged_append, paged_decode_attention
sk_kv4_unpack          kv4_unpack (+ kv4_row_bytes)
sk_paged_reserve, sk_paged_fork, sk_paged_compact
                       PagedGroup
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsinkkv.so")

SK_OK, SK_ERR_ARG, SK_ERR_CAPACITY, SK_ERR_POSITION_RANGE, SK_ERR_UNSUPPORTED, SK_ERR_CUDA = range(6)
SK_BF16, SK_F32, SK_I8, SK_I4 = 0, 1, 2, 3
SK_LAYER_RING, SK_LAYER_GLOBAL = 0, 1
SK_DEVERR_POSITION_RANGE, SK_DEVERR_CAPACITY, SK_DEVERR_TIMEOUT, SK_DEVERR_BLOCK_TABLE = 1, 2, 4, 8
SK_DEVERR_STATE = 16


class SinkKVError(RuntimeError):
    """A non-OK sk_status from the library."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_lib().sk_status_str(status).decode()}")


class RopeConfig(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("neox", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("theta", ctypes.c_double), ("yarn_factor", ctypes.c_double),
                ("yarn_orig_ctx", ctypes.c_int64), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("max_positions", ctypes.c_int64)]


class KVLayerStruct(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("k_dtype", ctypes.c_int32), ("v_dtype", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("window", ctypes.c_int32), ("capacity", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("head", ctypes.c_void_p), ("count", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("err", ctypes.c_void_p)]


class PagedLayerStruct(ctypes.Structure):
    _fields_ = [("k_dtype", ctypes.c_int32), ("v_dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("n_sink_blocks", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("window", ctypes.c_int32), ("n_blocks", ctypes.c_int64), ("k_pool", ctypes.c_void_p),
                ("v_pool", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("sink_block_ids", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("err", ctypes.c_void_p)]


_LIB = None

# (name, restype, argtypes) of every entry point in include/sinkkv.h
_SIGNATURES = [
    ("sk_rope_table_create", ctypes.c_int, [ctypes.POINTER(RopeConfig), ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]),
    ("sk_rope_table_rebuild", ctypes.c_int, [ctypes.c_void_p, ctypes.c_double, ctypes.c_void_p]),
    ("sk_rope_table_destroy", None, [ctypes.c_void_p]),
    ("sk_rope_table_info", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(RopeConfig), ctypes.POINTER(ctypes.c_void_p)]),
    ("sk_rope_table_fill_host", ctypes.c_int, [ctypes.POINTER(RopeConfig), ctypes.c_int32, ctypes.c_void_p]),
    ("sk_rope_dynamic_factor", ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_double, ctypes.c_double,
                                              ctypes.POINTER(ctypes.c_double)]),
    ("sk_rope_dynamic_create", ctypes.c_int, [ctypes.POINTER(RopeConfig), ctypes.c_double, ctypes.c_double,
                                              ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]),
    ("sk_rope_dynamic_table", ctypes.c_void_p, [ctypes.c_void_p]),
    ("sk_rope_dynamic_current_factor", ctypes.c_double, [ctypes.c_void_p]),
    ("sk_rope_dynamic_update", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(KVLayerStruct),
                                              ctypes.c_int32, ctypes.c_void_p, ctypes.POINTER(ctypes.c_double),
                                              ctypes.POINTER(ctypes.c_int32)]),
    ("sk_rope_dynamic_destroy", None, [ctypes.c_void_p]),
    ("sk_rope_apply", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                     ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    ("sk_kv_append", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(KVLayerStruct), ctypes.c_void_p, ctypes.c_int32,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]),
    ("sk_decode_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(KVLayerStruct), ctypes.c_int32]),
    ("sk_decode_attention", ctypes.c_int, [ctypes.POINTER(KVLayerStruct), ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                           ctypes.c_void_p]),
    ("sk_decode_attention_noalloc", ctypes.c_int, [ctypes.POINTER(KVLayerStruct), ctypes.c_void_p, ctypes.c_int32,
                                                   ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    ("sk_decode_step_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(KVLayerStruct), ctypes.c_int32]),
    ("sk_decode_step", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(KVLayerStruct), ctypes.c_void_p, ctypes.c_int32,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    ("sk_prefill_prior_keys", ctypes.c_int64, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]),
    ("sk_selftest_bounded_wait", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    ("sk_selftest_prefill_stall", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                                 ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32,
                                                 ctypes.c_void_p, ctypes.c_void_p]),
    ("sk_prefill_workspace_bytes", ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                     ctypes.c_int64]),
    ("sk_prefill_attention", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                            ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                            ctypes.POINTER(KVLayerStruct), ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                            ctypes.c_void_p]),
    ("sk_kv_rerotate", ctypes.c_int, [ctypes.POINTER(KVLayerStruct), ctypes.c_int32, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    ("sk_paged_append", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(PagedLayerStruct), ctypes.c_void_p,
                                       ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                       ctypes.c_int32, ctypes.c_void_p]),
    ("sk_paged_decode_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(PagedLayerStruct), ctypes.c_int32]),
    ("sk_paged_decode_attention", ctypes.c_int, [ctypes.POINTER(PagedLayerStruct), ctypes.c_void_p, ctypes.c_int32,
                                                 ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_size_t, ctypes.c_void_p]),
    ("sk_kv_shift_recent", ctypes.c_int, [ctypes.POINTER(KVLayerStruct), ctypes.c_int32, ctypes.c_void_p,
                                          ctypes.c_int32, ctypes.c_void_p]),
    ("sk_paged_pages_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(PagedLayerStruct)]),
    ("sk_paged_reserve", ctypes.c_int, [ctypes.POINTER(PagedLayerStruct), ctypes.c_int32, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    ("sk_paged_fork", ctypes.c_int, [ctypes.POINTER(PagedLayerStruct), ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p]),
    ("sk_paged_compact", ctypes.c_int, [ctypes.POINTER(PagedLayerStruct), ctypes.c_int32, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    ("sk_kv4_unpack", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    ("sk_sync_check", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.POINTER(ctypes.c_uint32)]),
    ("sk_status_str", ctypes.c_char_p, [ctypes.c_int]),
    ("sk_version", ctypes.c_int32, []),
]

EXPORTED = [name for name, _, _ in _SIGNATURES]


def _lib():
    """Load libsinkkv.so once; raise loudly if it is missing (no fallback)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libsinkkv.so not built at {LIB_PATH}; run "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, res, args in _SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _check(status: int, what: str):
    if status != SK_OK:
        raise SinkKVError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    """The cudaStream_t of a torch stream, or of the current one (read without making a
    stream object where torch offers that: a call's marshalling is most of a short one)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and torch.cuda.is_initialized():
        return _raw_stream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_SK_DTYPES = {torch.bfloat16: SK_BF16, torch.float32: SK_F32, torch.int8: SK_I8,
              torch.uint8: SK_I4}  # uint8: rows of 4-bit codes and their parameters


def _sk_dtype(dt: torch.dtype) -> int:
    d = _SK_DTYPES.get(dt)
    if d is None:
        raise TypeError(f"unsupported dtype {dt}")
    return d


def kv4_row_bytes(head_dim: int) -> int:
    """Bytes of a 4-bit cache row, K and V of one token and kv head (SK_KV4_ROW_BYTES)."""
    return head_dim + head_dim // 4


def _kv4_head_dim(row_bytes: int) -> int:
    if row_bytes % 5:
        raise ValueError("rows are not 4-bit cache rows")
    return row_bytes // 5 * 4


def _row_head_dim(k: torch.Tensor) -> int:
    """head_dim of a cache buffer [..., row]: its last size, or that of 4-bit rows."""
    return _kv4_head_dim(k.shape[-1]) if k.dtype == torch.uint8 else k.shape[-1]


def _need_contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


# ---------------------------------------------------------------------------
# RoPE table
# ---------------------------------------------------------------------------

class RopeTable:
    """Library-owned cos/sin table (sk_rope_table_create / rebuild / destroy)."""

    def __init__(self, head_dim: int, rotary_dim: int, theta: float, max_positions: int,
                 neox: bool = True, yarn_factor: float = 1.0, yarn_orig_ctx: int = 4096,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, stream=None):
        self.cfg = RopeConfig(head_dim, rotary_dim, 1 if neox else 0, 0, float(theta),
                              float(yarn_factor), int(yarn_orig_ctx), float(beta_fast),
                              float(beta_slow), int(max_positions))
        h = ctypes.c_void_p()
        _check(_lib().sk_rope_table_create(ctypes.byref(self.cfg), _stream(stream), ctypes.byref(h)),
               "sk_rope_table_create")
        self.handle = h

    def rebuild(self, yarn_factor: float, stream=None):
        _check(_lib().sk_rope_table_rebuild(self.handle, float(yarn_factor), _stream(stream)),
               "sk_rope_table_rebuild")
        self.cfg.yarn_factor = float(yarn_factor)

    def device_ptr(self) -> int:
        out = ctypes.c_void_p()
        _check(_lib().sk_rope_table_info(self.handle, None, ctypes.byref(out)), "sk_rope_table_info")
        return out.value

    def config(self) -> RopeConfig:
        c = RopeConfig()
        _check(_lib().sk_rope_table_info(self.handle, ctypes.byref(c), None), "sk_rope_table_info")
        return c

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _lib().sk_rope_table_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def rope_table_fill_host(head_dim: int, rotary_dim: int, theta: float, max_positions: int, neox: bool = True,
                         yarn_factor: float = 1.0, yarn_orig_ctx: int = 4096, beta_fast: float = 32.0,
                         beta_slow: float = 1.0, n_threads: int = 0):
    """The table as sk_rope_table_fill_host builds it on the host (no device):
    numpy float32 [max_positions, rotary_dim/2, 2] of (cos, sin) pairs."""
    import numpy as np
    cfg = RopeConfig(head_dim, rotary_dim, 1 if neox else 0, 0, float(theta), float(yarn_factor),
                     int(yarn_orig_ctx), float(beta_fast), float(beta_slow), int(max_positions))
    out = np.empty((max_positions, rotary_dim // 2, 2), dtype=np.float32)
    _check(_lib().sk_rope_table_fill_host(ctypes.byref(cfg), int(n_threads), out.ctypes.data_as(ctypes.c_void_p)),
           "sk_rope_table_fill_host")
    return out


def dynamic_factor(total_positions: int, orig_ctx: int, step: float = 0.125, cap: float = 2.0) -> float:
    """The YaRN factor for a dialog of total_positions (sk_rope_dynamic_factor)."""
    f = ctypes.c_double()
    _check(_lib().sk_rope_dynamic_factor(int(total_positions), int(orig_ctx), float(step), float(cap),
                                         ctypes.byref(f)), "sk_rope_dynamic_factor")
    return f.value


class _TableView(RopeTable):
    """A table owned by another library object (not freed here)."""

    def __init__(self, handle: int, owner):
        self.handle = ctypes.c_void_p(handle)
        self._owner = owner
        self.cfg = self.config()

    def rebuild(self, yarn_factor: float, stream=None):
        raise RuntimeError("the table of a DynamicRope changes only through DynamicRope.update")

    def close(self):
        self.handle = ctypes.c_void_p()


class DynamicRope:
    """A RoPE table whose YaRN factor follows the dialog's length (sk_rope_dynamic_*).
    ``table`` is the live table to pass to kv_append / rope_apply; ``update`` picks the
    factor for a length and, on a change, turns the given layers' cached keys."""

    def __init__(self, head_dim: int, rotary_dim: int, theta: float, max_positions: int, orig_ctx: int,
                 neox: bool = True, yarn_factor: float = 1.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 step: float = 0.125, cap: float = 0.0, stream=None):
        cfg = RopeConfig(head_dim, rotary_dim, 1 if neox else 0, 0, float(theta), float(yarn_factor),
                         int(orig_ctx), float(beta_fast), float(beta_slow), int(max_positions))
        h = ctypes.c_void_p()
        _check(_lib().sk_rope_dynamic_create(ctypes.byref(cfg), float(step), float(cap), _stream(stream),
                                             ctypes.byref(h)), "sk_rope_dynamic_create")
        self.handle = h
        self.table = _TableView(_lib().sk_rope_dynamic_table(h), self)

    @property
    def factor(self) -> float:
        return float(_lib().sk_rope_dynamic_current_factor(self.handle))

    def update(self, total_positions: int, layers: Sequence["KVLayer"] = (), stream=None):
        """Returns (factor now in force, whether it changed)."""
        arr = (KVLayerStruct * max(1, len(layers)))(*[L.struct() for L in layers])
        f = ctypes.c_double()
        sw = ctypes.c_int32()
        _check(_lib().sk_rope_dynamic_update(self.handle, int(total_positions), arr, len(layers), _stream(stream),
                                             ctypes.byref(f), ctypes.byref(sw)), "sk_rope_dynamic_update")
        return f.value, bool(sw.value)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            self.table.close()
            _lib().sk_rope_dynamic_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# KV layer (caller-owned device buffers held as torch tensors)
# ---------------------------------------------------------------------------

@dataclass
class KVLayer:
    """One layer's cache for a batch, as described by sk_kv_layer.

    k, v: [batch, n_kv_heads, capacity, head_dim]; k_scale: [batch, n_kv_heads, capacity]
    float32 (int8 K only); head, count: int32 [batch] (ring); pos: int64 [batch];
    err: uint32 word as int32 [1].  A 4-bit cache: k is uint8 [batch, n_kv_heads,
    capacity, kv4_row_bytes(head_dim)], rows of K and V together, and v is None.
    """
    kind: int
    k: torch.Tensor
    v: Optional[torch.Tensor]
    pos: torch.Tensor
    sinks: int = 0
    window: int = 0
    head: Optional[torch.Tensor] = None
    count: Optional[torch.Tensor] = None
    k_scale: Optional[torch.Tensor] = None
    err: Optional[torch.Tensor] = None

    @staticmethod
    def allocate(kind: int, batch: int, n_kv_heads: int, head_dim: int, *, sinks: int = 0,
                 window: int = 0, capacity: Optional[int] = None, k_dtype=torch.bfloat16,
                 v_dtype=torch.bfloat16, device="cuda", with_v: bool = True,
                 bits: Optional[int] = None) -> "KVLayer":
        """with_v=False leaves V as a one-row placeholder, for callers (such as a
        key rerotation) that never touch V.  bits=4: a 4-bit cache (k_dtype, v_dtype and
        with_v do not apply)."""
        if bits not in (None, 4):
            raise ValueError("bits must be 4 (or None: a cache of k_dtype and v_dtype)")
        if kind == SK_LAYER_RING:
            capacity = sinks + window
        assert capacity is not None and capacity >= 1
        if bits == 4:
            k_dtype, row = torch.uint8, kv4_row_bytes(head_dim)
        else:
            row = head_dim
        k = torch.zeros(batch, n_kv_heads, capacity, row, dtype=k_dtype, device=device)
        v = None if bits == 4 else (torch.zeros(batch, n_kv_heads, capacity, head_dim, dtype=v_dtype, device=device) if with_v
             else torch.zeros(1, 1, 1, head_dim, dtype=v_dtype, device=device))
        ks = (torch.ones(batch, n_kv_heads, capacity, dtype=torch.float32, device=device)
              if k_dtype == torch.int8 else None)
        z32 = lambda: torch.zeros(batch, dtype=torch.int32, device=device)
        return KVLayer(kind, k, v, torch.zeros(batch, dtype=torch.int64, device=device), sinks, window,
                       z32() if kind == SK_LAYER_RING else None, z32() if kind == SK_LAYER_RING else None,
                       ks, torch.zeros(1, dtype=torch.int32, device=device))

    @property
    def batch(self):
        return self.k.shape[0]

    @property
    def n_kv_heads(self):
        return self.k.shape[1]

    @property
    def capacity(self):
        return self.k.shape[2]

    @property
    def head_dim(self):
        return _row_head_dim(self.k)

    def struct(self) -> KVLayerStruct:
        k, v, ks, head, count, pos, err = (self.k, self.v, self.k_scale, self.head, self.count, self.pos,
                                           self.err)
        _need_contig(k, v, ks, head, count, pos)
        kd = _sk_dtype(k.dtype)
        B, H, cap, D = k.shape
        return KVLayerStruct(self.kind, kd, kd if v is None else _sk_dtype(v.dtype), B, H,
                             _kv4_head_dim(D) if kd == SK_I4 else D, self.sinks, self.window, cap, k.data_ptr(),
                             None if v is None else v.data_ptr(), None if ks is None else ks.data_ptr(),
                             None if head is None else head.data_ptr(), None if count is None else count.data_ptr(),
                             pos.data_ptr(), None if err is None else err.data_ptr())

    def error_bits(self) -> int:
        """Read the device error word (synchronises)."""
        return 0 if self.err is None else int(self.err.item()) & 0xFFFFFFFF


# ---------------------------------------------------------------------------
# Entry points
# ---------------------------------------------------------------------------

def rope_apply(table: RopeTable, x: torch.Tensor, positions: torch.Tensor,
               err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotate x [n_tok, H, D] in place at positions [n_tok] (sk_rope_apply)."""
    _need_contig(x, positions)
    n_tok, H = x.shape[0], x.shape[1]
    _check(_lib().sk_rope_apply(table.handle, _ptr(x), _sk_dtype(x.dtype), n_tok, H, _ptr(positions),
                                _ptr(err), _stream(stream)), "sk_rope_apply")
    return x


def kv_append(table: Optional[RopeTable], layer: KVLayer, q: Optional[torch.Tensor], k: torch.Tensor,
              v: torch.Tensor, stream=None):
    """Fused RoPE + append of T tokens per sequence (sk_kv_append).

    q [B, T, Hq, D] (optional) and k [B, T, Hkv, D] are rotated in place; v [B, T, Hkv, D].
    table None: k is already rotated and is appended as given (q must be None)."""
    _need_contig(q, k, v)
    T = k.shape[1]
    hq = 0 if q is None else q.shape[2]
    s = layer.struct()
    _check(_lib().sk_kv_append(None if table is None else table.handle, ctypes.byref(s), _ptr(q), hq, _ptr(k),
                               _ptr(v),
                               _sk_dtype(k.dtype), T, _stream(stream)), "sk_kv_append")


def decode_workspace_bytes(layer: KVLayer, n_q_heads: int) -> int:
    s = layer.struct()
    return int(_lib().sk_decode_workspace_bytes(ctypes.byref(s), n_q_heads))


def _sink_logits(sink_logits: Optional[torch.Tensor], n_q_heads: int):
    """Checks learned sink logits (float32 [n_q_heads] on the device, or None)."""
    if sink_logits is None:
        return None
    if sink_logits.dtype != torch.float32 or sink_logits.numel() != n_q_heads or not sink_logits.is_contiguous():
        raise ValueError("sink_logits must be a contiguous float32 tensor of n_q_heads values")
    return _ptr(sink_logits)


def decode_attention(layer: KVLayer, q_rot: torch.Tensor, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None,
                     sink_logits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Split-K decode attention of q_rot [B, Hq, D] over the layer's visible set;
    optional learned per-head sink logits (float32 [Hq], clamped to [-10, 15])."""
    _need_contig(q_rot)
    Hq = q_rot.shape[1]
    if out is None:
        out = torch.empty_like(q_rot)
    lib, s = _lib(), layer.struct()
    ref = ctypes.byref(s)
    need = lib.sk_decode_workspace_bytes(ref, Hq)
    if need == 0:
        raise SinkKVError(SK_ERR_UNSUPPORTED, "sk_decode_workspace_bytes")
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if size < need:
        size, workspace = need, torch.empty(need, dtype=torch.uint8, device=q_rot.device)
    _check(lib.sk_decode_attention(ref, q_rot.data_ptr(), Hq, _sk_dtype(q_rot.dtype),
                                   _sink_logits(sink_logits, Hq), out.data_ptr(), workspace.data_ptr(), size,
                                   _stream(stream)), "sk_decode_attention")
    return out


def decode_attention_noalloc(layer: KVLayer, q_rot: torch.Tensor, out: torch.Tensor, stream=None,
                             sink_logits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode attention for callers that cannot allocate device memory: the scratch
    is the library's fixed 4 MiB device array (sk_decode_attention_noalloc); `out`
    must be given.  Calls that may overlap on the GPU race on that array."""
    _need_contig(q_rot, out)
    s = layer.struct()
    _check(_lib().sk_decode_attention_noalloc(ctypes.byref(s), _ptr(q_rot), q_rot.shape[1],
                                              _sk_dtype(q_rot.dtype), _sink_logits(sink_logits, q_rot.shape[1]),
                                              _ptr(out), _stream(stream)),
           "sk_decode_attention_noalloc")
    return out


def decode_step_workspace_bytes(layer: KVLayer, n_q_heads: int) -> int:
    s = layer.struct()
    return int(_lib().sk_decode_step_workspace_bytes(ctypes.byref(s), n_q_heads))


def decode_step(table: Optional[RopeTable], layer: KVLayer, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
                sink_logits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode token per sequence: RoPE + append + attention in two kernels
    (sk_decode_step).  q [B, Hq, D], k and v [B, Hkv, D], unrotated and left as they are
    (unlike kv_append); returns out [B, Hq, D].  table None: q and k come rotated."""
    _need_contig(q, k, v)
    Hq = q.shape[1]
    if out is None:
        out = torch.empty_like(q)
    s = layer.struct()
    need = int(_lib().sk_decode_step_workspace_bytes(ctypes.byref(s), Hq))
    if need == 0:
        raise SinkKVError(SK_ERR_UNSUPPORTED, "sk_decode_step_workspace_bytes")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(_lib().sk_decode_step(None if table is None else table.handle, ctypes.byref(s), _ptr(q), Hq, _ptr(k),
                                 _ptr(v), _sk_dtype(q.dtype), _sink_logits(sink_logits, Hq), _ptr(out),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
           "sk_decode_step")
    return out


def prefill_prior_keys(p0: int, sinks: int, window: int) -> int:
    """Keys a chunk starting at p0 takes from a prior cache (sk_prefill_prior_keys)."""
    n = int(_lib().sk_prefill_prior_keys(int(p0), int(sinks), int(window)))
    if n < 0:
        raise SinkKVError(SK_ERR_ARG, "sk_prefill_prior_keys")
    return n


def prefill_workspace_bytes(batch: int, T: int, n_kv_heads: int, head_dim: int, prior_keys: int = 0) -> int:
    return int(_lib().sk_prefill_workspace_bytes(batch, T, n_kv_heads, head_dim, int(prior_keys)))


def prefill_attention(q_rot: torch.Tensor, k_rot: torch.Tensor, v: torch.Tensor, p0: int, sinks: int,
                      window: int, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      err: Optional[torch.Tensor] = None, stream=None,
                      sink_logits: Optional[torch.Tensor] = None,
                      prior: Optional["KVLayer"] = None) -> torch.Tensor:
    """Masked prefill attention of a chunk: q [B,T,Hq,D], k/v [B,T,Hkv,D]
    (sk_prefill_attention); window <= 0 is a global layer; optional learned per-head
    sink logits (float32 [Hq]); ``prior``: the layer whose cache holds positions
    [0, p0) of every sequence (the chunk not yet appended), whose keys the chunk then
    also sees."""
    _need_contig(q_rot, k_rot, v)
    B, T, Hq, D = q_rot.shape
    Hkv = k_rot.shape[2]
    if out is None:
        out = torch.empty_like(q_rot)
    prior_keys = prefill_prior_keys(p0, sinks, window) if prior is not None else 0
    need = prefill_workspace_bytes(B, T, Hkv, D, prior_keys)
    if need == 0:
        raise SinkKVError(SK_ERR_UNSUPPORTED, "sk_prefill_workspace_bytes")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_rot.device)
    ps = ctypes.byref(prior.struct()) if prior is not None else None
    _check(_lib().sk_prefill_attention(_ptr(q_rot), _ptr(k_rot), _ptr(v), B, T, Hq, Hkv, D, int(p0), int(sinks),
                                       int(window), ps, _sink_logits(sink_logits, Hq), _ptr(out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream)),
           "sk_prefill_attention")
    return out


def kv_rerotate(layers: Sequence[KVLayer], table_from: RopeTable, table_to: RopeTable, stream=None):
    """Turn every cached key of `layers` from table_from's factor to table_to's (sk_kv_rerotate)."""
    arr = (KVLayerStruct * len(layers))(*[l.struct() for l in layers])
    _check(_lib().sk_kv_rerotate(arr, len(layers), table_from.handle, table_to.handle, _stream(stream)),
           "sk_kv_rerotate")


@dataclass
class PagedLayer:
    """A paged layer's caller-owned device buffers (sk_paged_layer): pools
    [n_blocks, H_kv, block_size, D], block_table int32 [B, max_blocks] (-1 = no block),
    sink_block_ids int32 [n_sink_blocks], seq_lens int64 [B].  A 4-bit cache: k_pool is
    uint8 [n_blocks, H_kv, block_size, kv4_row_bytes(D)] and v_pool is None."""
    k_pool: torch.Tensor
    v_pool: Optional[torch.Tensor]
    block_table: torch.Tensor
    sink_block_ids: Optional[torch.Tensor]
    seq_lens: torch.Tensor
    err: torch.Tensor
    sinks: int
    window: int

    @staticmethod
    def allocate(batch: int, n_kv_heads: int, head_dim: int, *, block_size: int, n_blocks: int, max_blocks: int,
                 sinks: int = 0, window: int = 0, n_sink_blocks: int = 0, dtype=torch.bfloat16,
                 device="cuda", bits: Optional[int] = None) -> "PagedLayer":
        """bits=4: a 4-bit cache (dtype does not apply)."""
        if bits not in (None, 4):
            raise ValueError("bits must be 4 (or None: a cache of dtype)")
        z = dict(dtype=dtype if bits is None else torch.uint8, device=device)
        row = head_dim if bits is None else kv4_row_bytes(head_dim)
        return PagedLayer(
            k_pool=torch.zeros(n_blocks, n_kv_heads, block_size, row, **z),
            v_pool=torch.zeros(n_blocks, n_kv_heads, block_size, row, **z) if bits is None else None,
            block_table=torch.full((batch, max_blocks), -1, dtype=torch.int32, device=device),
            sink_block_ids=(torch.arange(n_sink_blocks, dtype=torch.int32, device=device)
                            if n_sink_blocks > 0 else None),
            seq_lens=torch.zeros(batch, dtype=torch.int64, device=device),
            err=torch.zeros(1, dtype=torch.int32, device=device), sinks=sinks, window=window)

    @property
    def batch(self):
        return self.block_table.shape[0]

    @property
    def n_kv_heads(self):
        return self.k_pool.shape[1]

    @property
    def block_size(self):
        return self.k_pool.shape[2]

    def struct(self) -> PagedLayerStruct:
        k, v, table, sinks = self.k_pool, self.v_pool, self.block_table, self.sink_block_ids
        kd = _sk_dtype(k.dtype)
        n_blocks, H, bs, D = k.shape
        B, max_blocks = table.shape
        return PagedLayerStruct(kd, kd if v is None else _sk_dtype(v.dtype), B, H,
                                _kv4_head_dim(D) if kd == SK_I4 else D, bs, max_blocks,
                                0 if sinks is None else sinks.numel(), self.sinks, self.window, n_blocks,
                                k.data_ptr(), None if v is None else v.data_ptr(), table.data_ptr(),
                                None if sinks is None else sinks.data_ptr(), self.seq_lens.data_ptr(),
                                self.err.data_ptr())

    def error_bits(self) -> int:
        return int(self.err.item())


def paged_append(table: RopeTable, layer: PagedLayer, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                 stream=None):
    """RoPE on q (optional) and k in place, then k, v into the pool slots of the block
    table (sk_paged_append); q [B, T, Hq, D], k/v [B, T, Hkv, D]."""
    _need_contig(k, v)
    if q is not None:
        _need_contig(q)
    s = layer.struct()
    _check(_lib().sk_paged_append(table.handle, ctypes.byref(s), _ptr(q), 0 if q is None else q.shape[2], _ptr(k),
                                  _ptr(v), _sk_dtype(k.dtype), k.shape[1], _stream(stream)), "sk_paged_append")


def paged_decode_workspace_bytes(layer: PagedLayer, n_q_heads: int) -> int:
    s = layer.struct()
    return int(_lib().sk_paged_decode_workspace_bytes(ctypes.byref(s), n_q_heads))


def paged_decode_attention(layer: PagedLayer, q_rot: torch.Tensor, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None,
                           sink_logits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode attention of q_rot [B, Hq, D] over a paged layer (sk_paged_decode_attention)."""
    _need_contig(q_rot)
    Hq = q_rot.shape[1]
    if out is None:
        out = torch.empty_like(q_rot)
    lib, s = _lib(), layer.struct()
    ref = ctypes.byref(s)
    need = lib.sk_paged_decode_workspace_bytes(ref, Hq)
    if need == 0:
        raise SinkKVError(SK_ERR_UNSUPPORTED, "sk_paged_decode_workspace_bytes")
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if size < need:
        size, workspace = need, torch.empty(need, dtype=torch.uint8, device=q_rot.device)
    _check(lib.sk_paged_decode_attention(ref, q_rot.data_ptr(), Hq, _sk_dtype(q_rot.dtype),
                                         _sink_logits(sink_logits, Hq), out.data_ptr(), workspace.data_ptr(), size,
                                         _stream(stream)), "sk_paged_decode_attention")
    return out


class PagedGroup:
    """The blocks of paged layers that share one block table (sk_paged_reserve / fork /
    compact).  ``ref``: int32 [n_blocks] uses of each block (default: an empty pool, with
    one use for each static sink block, whose ids are then read from the device).  The
    group works on the tensors that the layers hold when it is made; replacing one of them
    takes a new group.  It owns one workspace: calls of one group on several streams must
    be ordered (they change the same table anyway)."""

    def __init__(self, layers: Sequence[PagedLayer], ref: Optional[torch.Tensor] = None):
        if len(layers) == 0:
            raise ValueError("a group needs a layer")
        self.layers = list(layers)
        L = self.layers[0]
        dev, n_blocks = L.k_pool.device, L.k_pool.shape[0]
        if ref is None:
            ref = torch.zeros(n_blocks, dtype=torch.int32, device=dev)
            if L.sink_block_ids is not None:
                ref[L.sink_block_ids.long()] = 1
        _check_i32("ref", ref, n_blocks, dev)
        self.ref = ref
        for x in self.layers:
            _need_contig(x.k_pool, x.v_pool, x.block_table, x.seq_lens)
            if x.block_table.dtype != torch.int32 or x.seq_lens.dtype != torch.int64:
                raise ValueError("block_table must be int32 and seq_lens int64")
            if x.seq_lens.numel() != x.batch:
                raise ValueError("seq_lens must hold a length for each request")
        self._structs = (PagedLayerStruct * len(self.layers))(*[x.struct() for x in self.layers])
        self._tensors = [(x.k_pool, x.v_pool, x.block_table, x.sink_block_ids, x.seq_lens, x.err) for x in self.layers]
        need = int(_lib().sk_paged_pages_workspace_bytes(self._structs))
        if need == 0:
            raise SinkKVError(SK_ERR_UNSUPPORTED, "sk_paged_pages_workspace_bytes")
        self._ws = torch.empty(need, dtype=torch.uint8, device=dev)

    @property
    def batch(self):
        return self.layers[0].batch

    def reserve(self, n_new: Optional[torch.Tensor] = None, granted: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """Blocks for n_new[b] new tokens of each request (int32 [batch]; None: one each).
        Returns granted, int32 [batch]: 1 where the request may append."""
        dev = self.ref.device
        if n_new is not None:
            _check_i32("n_new", n_new, self.batch, dev)
        if granted is None:
            granted = torch.empty(self.batch, dtype=torch.int32, device=dev)
        else:
            _check_i32("granted", granted, self.batch, dev)
        _check(_lib().sk_paged_reserve(self._structs, len(self.layers), _ptr(self.ref), _ptr(n_new), _ptr(granted),
                                       _ptr(self._ws), self._ws.numel(), _stream(stream)), "sk_paged_reserve")
        return granted

    def fork(self, parents: torch.Tensor, stream=None):
        """Request b continues from request parents[b] (int32 [batch]; b: stays, -1: released)."""
        _check_i32("parents", parents, self.batch, self.ref.device)
        _check(_lib().sk_paged_fork(self._structs, len(self.layers), _ptr(self.ref), _ptr(parents), _stream(stream)),
               "sk_paged_fork")

    def compact(self, block_map: Optional[torch.Tensor] = None, stream=None):
        """Blocks in use to the lowest ids.  Returns (block_map int32 [n_blocks]: new ids, -1
        for blocks that were free; used int32 [1]: one past the highest id in use)."""
        dev = self.ref.device
        if block_map is None:
            block_map = torch.empty_like(self.ref)
        else:
            _check_i32("block_map", block_map, self.ref.numel(), dev)
        used = torch.empty(1, dtype=torch.int32, device=dev)
        _check(_lib().sk_paged_compact(self._structs, len(self.layers), _ptr(self.ref), _ptr(block_map), _ptr(used),
                                       _ptr(self._ws), self._ws.numel(), _stream(stream)), "sk_paged_compact")
        return block_map, used


def _check_i32(name: str, t: torch.Tensor, n: int, device):
    if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} values on {device}")


def kv4_unpack(rows: torch.Tensor, dtype=torch.bfloat16, stream=None):
    """The values that 4-bit cache rows stand for (sk_kv4_unpack): rows uint8 [..., row bytes]
    (a 4-bit KVLayer's k, a PagedLayer's k_pool, or any contiguous run of their rows) ->
    K, V of dtype (bf16 or fp32) [..., head_dim]."""
    if rows.dtype != torch.uint8:
        raise TypeError("rows must be uint8")
    _need_contig(rows)
    D = _row_head_dim(rows)
    K = torch.empty(*rows.shape[:-1], D, dtype=dtype, device=rows.device)
    V = torch.empty_like(K)
    _check(_lib().sk_kv4_unpack(_ptr(rows), rows.numel() // rows.shape[-1], D, _ptr(K), _ptr(V), _sk_dtype(dtype),
                                _stream(stream)), "sk_kv4_unpack")
    return K, V


def kv_shift_recent(layers: Sequence[KVLayer], table: RopeTable, delta: int, stream=None):
    """Turn the recent keys of ring layers by `delta` positions in place; sinks and
    values stay (sk_kv_shift_recent)."""
    arr = (KVLayerStruct * max(1, len(layers)))(*[L.struct() for L in layers])
    _check(_lib().sk_kv_shift_recent(arr, len(layers), table.handle, int(delta), _stream(stream)),
           "sk_kv_shift_recent")


def sync_check(err: torch.Tensor, clear: bool = False, stream=None):
    """(status, bits) of a device error word after the queued work (sk_sync_check)."""
    bits = ctypes.c_uint32()
    st = _lib().sk_sync_check(_ptr(err), 1 if clear else 0, _stream(stream), ctypes.byref(bits))
    return int(st), int(bits.value)


def selftest_bounded_wait(err: torch.Tensor, stream=None) -> None:
    """Launch the bounded-wait diagnostic (sk_selftest_bounded_wait): about one second
    later SK_DEVERR_TIMEOUT is set in `err`."""
    _check(_lib().sk_selftest_bounded_wait(_ptr(err), _stream(stream)), "sk_selftest_bounded_wait")


def selftest_prefill_stall(q_rot: torch.Tensor, k_rot: torch.Tensor, v: torch.Tensor, stall_tile: int,
                           err: torch.Tensor, stream=None) -> torch.Tensor:
    """Run the prefill pipeline on a global causal chunk whose P of tile `stall_tile` is
    never signalled ready (sk_selftest_prefill_stall): the blocks that reach it give up
    after about one second and set SK_DEVERR_TIMEOUT in `err`.  Returns the (undefined)
    output buffer."""
    _need_contig(q_rot, k_rot, v)
    B, T, Hq, D = q_rot.shape
    Hkv = k_rot.shape[2]
    out = torch.empty_like(q_rot)
    need = prefill_workspace_bytes(B, T, Hkv, D, 0)
    if need == 0:
        raise SinkKVError(SK_ERR_UNSUPPORTED, "sk_prefill_workspace_bytes")
    ws = torch.empty(need, dtype=torch.uint8, device=q_rot.device)
    _check(_lib().sk_selftest_prefill_stall(_ptr(q_rot), _ptr(k_rot), _ptr(v), B, T, Hq, Hkv, D, _ptr(out), _ptr(ws),
                                            need, int(stall_tile), _ptr(err), _stream(stream)),
           "sk_selftest_prefill_stall")
    return out


def version() -> int:
    return int(_lib().sk_version())
