"""Thin ctypes binding of libqasa (see include/qasa.h for every contract).

Argument marshalling only: torch tensors supply device memory and the current
CUDA stream; every step of the computation runs in the library's kernels.
Importing this module loads ``libqasa.so``; a missing library raises at once
(there is no fallback path).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import Optional, Sequence, Tuple, Union

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqasa.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError("libqasa.so is not built (run query_aware_sparse_append_gb300.build.build())")
_lib = ctypes.CDLL(_LIB_PATH)

DTYPE_IDS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
E4M3 = 3            # FP8 KV: uint8 pools and boxes holding E4M3 codes, plus page_scales
STATUS_OK = 0

DEVERR = {
    0x1: "page id out of range",
    0x2: "seq_len out of range",
    0x4: "budget above max_budget",
    0x8: "bounded wait timed out",
    0x10: "append length out of range",
    0x20: "selected id out of range",
    0x40: "position beyond the rotation table",
    0x80: "parent out of range",
    0x100: "kept tokens not ascending within the sequence",
}


class _Cache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("page_bounds", ctypes.c_void_p), ("num_phys_pages", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("page_scales", ctypes.c_void_p)]


class _Rotation(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("max_positions", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class _TokenRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


class _Positions(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("axis_stride", ctypes.c_int64), ("batch_stride", ctypes.c_int64),
                ("num_axes", ctypes.c_int32), ("pair_axes", ctypes.c_char_p)]


_ThreeRows = ctypes.c_int64 * 9      # three qasa_token_rows, filled at once


_P = ctypes.c_void_p
_I = ctypes.c_int32
_C = ctypes.POINTER(_Cache)
_lib.qasa_kv_append.argtypes = [_C, _P, _I, _P, _P, _P, _P, _I, _I, _P, _P]
_lib.qasa_kv_append.restype = _I
_lib.qasa_decode_workspace_size.argtypes = [_I, _I, _C, _I]
_lib.qasa_decode_workspace_size.restype = ctypes.c_size_t
_lib.qasa_select_pages.argtypes = [_C, _P, _I, _P, _I, _P, _P, _I, _P, _P, _P, ctypes.c_size_t, _I,
                                   _P, _P]
_lib.qasa_select_pages.restype = _I
_lib.qasa_sparse_attention.argtypes = [_C, _P, _I, _P, _I, _P, _P, _I, _P, ctypes.c_float, _P, _P,
                                       ctypes.c_size_t, _I, _P, _P]
_lib.qasa_sparse_attention.restype = _I
_lib.qasa_sparse_decode_attention.argtypes = [_C, _P, _I, _P, _I, _P, _P, _I, ctypes.c_float, _P,
                                              _P, _P, _P, ctypes.c_size_t, _I, _P, _P]
_lib.qasa_sparse_decode_attention.restype = _I
_lib.qasa_dense_decode_attention.argtypes = [_C, _P, _I, _P, _I, _P, ctypes.c_float, _P, _P,
                                             ctypes.c_size_t, _I, _P, _P]
_lib.qasa_dense_decode_attention.restype = _I
_lib.qasa_sparse_decode_attention_noalloc.argtypes = [_C, _P, _I, _P, _I, _P, _P, _I, ctypes.c_float,
                                                      _P, _P, _P, _I, _P, _P]
_lib.qasa_sparse_decode_attention_noalloc.restype = _I
_lib.qasa_kv_append_rotated.argtypes = [_C, _P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _I, _I, _P, _P]
_lib.qasa_kv_append_rotated.restype = _I
_lib.qasa_kv_append_positioned.argtypes = [_C, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _I, _I, _P, _P]
_lib.qasa_kv_append_positioned.restype = _I
_lib.qasa_kv_keep_tokens.argtypes = [_C, _P, _I, _P, _P, _P, _I, _P, _P, _I, _P, _P]
_lib.qasa_kv_keep_tokens.restype = _I
_lib.qasa_kv_copy_pages.argtypes = [_C, _P, _P, _I, _P, _P]
_lib.qasa_kv_copy_pages.restype = _I
_lib.qasa_kv_fork.argtypes = [_C, _P, _I, _P, _I, _P, _P, _I, _P, _P, _P, _P]
_lib.qasa_kv_fork.restype = _I
_lib.qasa_tree_workspace_size.argtypes = [_I, _I, _C, _I, _I]
_lib.qasa_tree_workspace_size.restype = ctypes.c_size_t
_lib.qasa_tree_attention.argtypes = [_C, _P, _I, _I, _P, _P, ctypes.c_int64, _P, _I, _P, _I, _I, ctypes.c_float, _P, _P,
                                     ctypes.c_size_t, _I, _P, _P]
_lib.qasa_tree_attention.restype = _I
_lib.qasa_tree_masks.argtypes = [_P, _I, _I, _P, _P, _P, _P, _P]
_lib.qasa_tree_masks.restype = _I
_lib.qasa_window_workspace_size.argtypes = [_I, _I, _C, _I, _I, _I, _I]
_lib.qasa_window_workspace_size.restype = ctypes.c_size_t
_lib.qasa_window_attention.argtypes = [_C, _P, _I, _I, _P, _P, _I, _P, _I, _I, ctypes.c_float, _P, _P, ctypes.c_size_t,
                                       _I, _P, _P]
_lib.qasa_window_attention.restype = _I
_lib.qasa_rebuild_page_bounds.argtypes = [_C, _P, _I, _P, _I, _P, _P]
_lib.qasa_rebuild_page_bounds.restype = _I
_lib.qasa_page_attention_mass.argtypes = [_C, _P, _I, _P, _I, _P, ctypes.c_float, _P, _I, _P, _P]
_lib.qasa_page_attention_mass.restype = _I
_lib.qasa_page_hit_rate.argtypes = [_C, _P, _I, _P, _P, _I, _P, _I, _P, _P, _P, _P, _P]
_lib.qasa_page_hit_rate.restype = _I
_lib.qasa_host_decode_workspace_size.argtypes = [_I, _I, _C, _I, _I]
_lib.qasa_host_decode_workspace_size.restype = ctypes.c_size_t
_lib.qasa_sparse_decode_attention_host.argtypes = [_C, _P, _I, _P, _I, _P, _P, _I, ctypes.c_float, _P, _P, _P,
                                                   ctypes.c_size_t, _I, _P, _P]
_lib.qasa_sparse_decode_attention_host.restype = _I
_lib.qasa_host_call_is_direct.argtypes = [_P] * 6
_lib.qasa_host_call_is_direct.restype = _I
_lib.qasa_status_string.argtypes = [_I]
_lib.qasa_status_string.restype = ctypes.c_char_p
_lib.qasa_version.restype = _I
_lib.qasa_debug_trace_bytes.restype = ctypes.c_size_t
_lib.qasa_debug_trace.argtypes = [_P, ctypes.c_size_t]
_lib.qasa_debug_trace.restype = _I

EXPORTED = ("qasa_kv_append", "qasa_decode_workspace_size", "qasa_select_pages",
            "qasa_sparse_attention", "qasa_sparse_decode_attention",
            "qasa_dense_decode_attention", "qasa_sparse_decode_attention_noalloc",
            "qasa_rebuild_page_bounds", "qasa_page_attention_mass", "qasa_page_hit_rate",
            "qasa_host_decode_workspace_size", "qasa_sparse_decode_attention_host",
            "qasa_host_call_is_direct", "qasa_kv_append_rotated", "qasa_window_workspace_size",
            "qasa_window_attention", "qasa_kv_append_positioned", "qasa_kv_keep_tokens", "qasa_kv_copy_pages",
            "qasa_kv_fork", "qasa_tree_workspace_size", "qasa_tree_attention", "qasa_tree_masks", "qasa_status_string", "qasa_version",
            "qasa_debug_trace_bytes", "qasa_debug_trace")

# trace buffer layout (include/qasa.h)
TRACE_MAX_CTAS = 4096
TRACE_SELECT_EVENTS = 4
TRACE_ATTN_EVENTS = 12


class QasaError(RuntimeError):
    pass


def library_path() -> str:
    return _LIB_PATH


def version() -> int:
    return int(_lib.qasa_version())


def debug_trace(buffer: Optional[torch.Tensor]) -> None:
    """Record per-CTA timestamps of every later selection and attention launch
    into `buffer` (a zeroed int64 device tensor of at least
    debug_trace_bytes() bytes); None turns recording off."""
    if buffer is None:
        _check(_lib.qasa_debug_trace(None, 0), "qasa_debug_trace")
        return
    _check(_lib.qasa_debug_trace(_ptr(buffer), buffer.numel() * buffer.element_size()), "qasa_debug_trace")


def debug_trace_bytes() -> int:
    return int(_lib.qasa_debug_trace_bytes())


def status_string(code: int) -> str:
    return _lib.qasa_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != STATUS_OK:
        raise QasaError("%s failed: %s (%d)" % (what, status_string(code), code))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


_HERE = contextlib.nullcontext()


def _allocating_on(stream: Optional[torch.cuda.Stream]):
    """Context whose tensors belong to the stream of a call: memory that the current stream gave back, and may
    still be working on, is not handed to a kernel on `stream`, nor theirs to the current stream while `stream`
    works on it."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _contig(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


class PagedKVCache:
    """Device pools of one attention layer (caller-owned memory, library layout).

    k_pool, v_pool : [num_phys_pages, num_kv_heads, page_size, head_dim]
    page_bounds    : [num_phys_pages, num_kv_heads, 2, head_dim]  (lo row, hi row)
    page_scales    : FP8 KV only (uint8 pools holding E4M3 codes):
                     [num_phys_pages, num_kv_heads, 4] float32 (amax of K, amax of V, -, -);
                     queries, outputs and appended K/V are then float16
    """

    def __init__(self, k_pool: torch.Tensor, v_pool: torch.Tensor, page_bounds: torch.Tensor,
                 page_scales: Optional[torch.Tensor] = None):
        if k_pool.shape != v_pool.shape or k_pool.dim() != 4:
            raise ValueError("k_pool and v_pool must share a 4-d shape")
        n, hkv, p, d = k_pool.shape
        if tuple(page_bounds.shape) != (n, hkv, 2, d):
            raise ValueError("page_bounds must be [num_phys_pages, num_kv_heads, 2, head_dim]")
        fp8 = k_pool.dtype == torch.uint8
        if not (k_pool.dtype == v_pool.dtype == page_bounds.dtype) or not (fp8 or k_pool.dtype in DTYPE_IDS):
            raise ValueError("pools must share one of float32 / float16 / bfloat16 / uint8 (E4M3 codes)")
        if fp8:
            if page_scales is None or tuple(page_scales.shape) != (n, hkv, 4) or page_scales.dtype != torch.float32:
                raise ValueError("FP8 pools need page_scales [num_phys_pages, num_kv_heads, 4] float32")
            _contig(page_scales, "page_scales")
        for t, nm in ((k_pool, "k_pool"), (v_pool, "v_pool"), (page_bounds, "page_bounds")):
            _contig(t, nm)
        self.k_pool, self.v_pool, self.page_bounds = k_pool, v_pool, page_bounds
        self.page_scales = page_scales if fp8 else None
        self.num_phys_pages, self.num_kv_heads, self.page_size, self.head_dim = n, hkv, p, d
        self.dtype = k_pool.dtype
        self.is_fp8 = fp8
        self.value_dtype = torch.float16 if fp8 else self.dtype     # of queries, outputs and appended values
        self.device_index = k_pool.get_device()                     # -1: not on a CUDA device
        self._c = _Cache(k_pool.data_ptr(), v_pool.data_ptr(), page_bounds.data_ptr(), n, hkv, p,
                         d, E4M3 if fp8 else DTYPE_IDS[k_pool.dtype],
                         page_scales.data_ptr() if fp8 else None)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, num_phys_pages: int, num_kv_heads: int, page_size: int, head_dim: int,
              dtype=torch.float16, device="cuda") -> "PagedKVCache":
        """dtype float32 / float16 / bfloat16, or torch.uint8 for FP8 (E4M3) KV."""
        shape = (num_phys_pages, num_kv_heads, page_size, head_dim)
        scales = (torch.zeros((num_phys_pages, num_kv_heads, 4), dtype=torch.float32, device=device)
                  if dtype == torch.uint8 else None)
        # K and V carved from one allocation (V right after K): the attention
        # kernel then fetches a page's K and V tiles with a single TMA box
        kv = torch.empty((2,) + shape, dtype=dtype, device=device)
        return cls(kv[0], kv[1],
                   torch.empty((num_phys_pages, num_kv_heads, 2, head_dim), dtype=dtype,
                               device=device), scales)

    @property
    def c_ref(self):
        return self._ref


def workspace_size(cache: PagedKVCache, batch: int, num_q_heads: int, max_pages_per_seq: int) -> int:
    return int(_lib.qasa_decode_workspace_size(batch, num_q_heads, cache.c_ref, max_pages_per_seq))


def alloc_workspace(cache: PagedKVCache, batch: int, num_q_heads: int, max_pages_per_seq: int,
                    device=None) -> torch.Tensor:
    n = workspace_size(cache, batch, num_q_heads, max_pages_per_seq)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or cache.k_pool.device)


def kv_append(cache: PagedKVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
              k_new: torch.Tensor, v_new: torch.Tensor, append_lens: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write k_new / v_new [B, T, Hkv, d] after seq_lens (not advanced) and update page boxes."""
    B, T = int(k_new.shape[0]), int(k_new.shape[1])
    _contig(k_new, "k_new"), _contig(v_new, "v_new"), _contig(block_table, "block_table")
    code = _lib.qasa_kv_append(cache.c_ref, _ptr(block_table), int(block_table.shape[1]),
                               _ptr(seq_lens), _ptr(append_lens), _ptr(k_new), _ptr(v_new), B, T,
                               _ptr(status), _stream(stream))
    _check(code, "qasa_kv_append")


# The stream and device lookups below are the ones behind torch.cuda.current_stream()
# and torch.cuda.current_device(), without the Stream object and the initialisation
# check: a decode step's append takes less time than those do.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)     # a torch without CUDA has neither
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _arg(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple, index: int):
    """Address of a contiguous tensor of this type and shape on CUDA device `index` (None: NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d" % (name, dtype, tuple(shape), index))


def _status_arg(status: Optional[torch.Tensor], index: int):
    if status is None:
        return None
    if status.dtype is torch.int32 and status.get_device() == index and status.numel() >= 1:
        return status.data_ptr()
    raise ValueError("status must be an int32 tensor on cuda:%d" % index)


def _token_rows(t: torch.Tensor, name: str, dtype: torch.dtype, head_dim: int, index: int) -> tuple:
    """The fields of a qasa_token_rows."""
    if t.dim() != 4 or t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be a %s tensor [batch, tokens, heads, head_dim] on cuda:%d" % (name, dtype, index))
    sb, st, sh, sc = t.stride()
    if (sc != 1 or sh != head_dim) and t.numel() and (sc != 1 or t.shape[2] > 1):
        raise ValueError("the heads of a token of %s must be contiguous" % name)
    return t.data_ptr(), sb, st


def _call_stream(stream: Optional[torch.cuda.Stream], index: int) -> int:
    """The stream of a call on device `index`: the one given, else the device's current one."""
    if stream is None:
        return _raw_stream(index)
    if stream.device_index != index:
        raise ValueError("stream and cache are on different devices")
    return stream.cuda_stream


def rotation_table(max_positions: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines of the angles pos * base^(-2 i / rot_dim), [max_positions, 2, rot_dim / 2]
    float32, computed in 64 bits (a far position's angle has few 32-bit digits left).  Any other
    table of this layout serves too (scaled or interpolated frequencies)."""
    freq = torch.pow(torch.tensor(float(base), dtype=torch.float64), -torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), 1).to(torch.float32).contiguous().to(device)


def kv_append_rotated(cache: PagedKVCache, block_table: torch.Tensor, seq_lens: torch.Tensor, k_new: torch.Tensor,
                      v_new: torch.Tensor, table: torch.Tensor, q: Optional[torch.Tensor] = None,
                      q_out: Optional[torch.Tensor] = None, append_lens: Optional[torch.Tensor] = None,
                      interleaved: bool = False, status: Optional[torch.Tensor] = None,
                      stream=None) -> Optional[torch.Tensor]:
    """kv_append with the position rotation applied on the way: k_new [B, T, Hkv, d] is rotated by the
    table's angles of its positions before it is stored, q [B, T, Hq, d] (optional) is rotated into
    q_out [B, T, Hq, d] (contiguous, allocated on the call's stream where not given, returned).  k_new, v_new and q may be
    parts of one tensor: any batch and token stride that is a multiple of 16 bytes.  table: as made by
    rotation_table, whose last dimension says how many channels turn; interleaved: neighbouring
    channels are the pairs (else channels rot_dim / 2 apart)."""
    index = cache.device_index
    if index >= 0 and _get_device() != index:
        with torch.cuda.device(index):
            return kv_append_rotated(cache, block_table, seq_lens, k_new, v_new, table, q, q_out, append_lens,
                                     interleaved, status, stream)
    return _append_rotated(cache, block_table, seq_lens, k_new, v_new, table, q, q_out, append_lens, interleaved, None, status,
                           stream)


def _append_rotated(cache, block_table, seq_lens, k_new, v_new, table, q, q_out, append_lens, interleaved, given, status,
                    stream):
    """The rotating append on the cache's device, the current one; `given`: (positions, pair_axes) or None."""
    index = cache.device_index
    value, d = cache.value_dtype, cache.head_dim
    kr = _token_rows(k_new, "k_new", value, d, index)
    vr = _token_rows(v_new, "v_new", value, d, index)
    shape = k_new.shape
    B, T, H, kd = shape
    if H != cache.num_kv_heads or kd != d or v_new.shape != shape:
        raise ValueError("k_new and v_new must be [batch, tokens, num_kv_heads, head_dim]")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages_per_seq]")
    maxp = block_table.shape[1]
    if table.dim() != 3 or table.shape[1] != 2:
        raise ValueError("table must be [max_positions, 2, rot_dim / 2]")
    positions, _, half = angles = table.shape
    rot = _Rotation(_arg(table, "table", torch.float32, angles, index), positions, 2 * half, 1 if interleaved else 0)
    qr, hq, out = (0, 0, 0), 0, None
    if q is not None:
        qr = _token_rows(q, "q", value, d, index)
        qb, qt, hq, qd = q.shape
        if qb != B or qt != T or qd != d:
            raise ValueError("q must have the batch and tokens of k_new and the cache's head_dim")
        if q_out is None:
            with _allocating_on(stream):
                q_out = torch.empty((B, T, hq, d), dtype=value, device=q.device)
        out = _arg(q_out, "q_out", value, (B, T, hq, d), index)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    rows = _ThreeRows(*kr, *vr, *qr)
    at = ctypes.addressof(rows)
    args = (
        _arg(block_table, "block_table", torch.int32, (B, maxp), index), maxp,
        _arg(seq_lens, "seq_lens", torch.int32, (B,), index), _arg(append_lens, "append_lens", torch.int32, (B,), index),
        None if q is None else at + 48, hq, out, at, at + 24, B, T, _status_arg(status, index), _call_stream(stream, index))
    if given is None:
        code = _lib.qasa_kv_append_rotated(cache.c_ref, ctypes.byref(rot), *args)
        if code:
            _check(code, "qasa_kv_append_rotated")
        return q_out
    pos = _positions(*given, B, T, half, index)
    code = _lib.qasa_kv_append_positioned(cache.c_ref, ctypes.byref(rot), ctypes.byref(pos), *args)
    if code:
        _check(code, "qasa_kv_append_positioned")
    return q_out


def _positions(positions: torch.Tensor, axes, B: int, T: int, half: int, index: int) -> _Positions:
    shape = positions.shape
    num = shape[0] if len(shape) == 3 else 1
    if len(shape) not in (2, 3) or positions.dtype is not torch.int32 or positions.get_device() != index \
            or shape[-1] != T or shape[-2] not in (1, B) or (T > 1 and positions.stride(-1) != 1):
        raise ValueError("positions must be an int32 tensor [axes, batch or 1, tokens] or [batch or 1, tokens] on cuda:%d, "
                         "its tokens contiguous" % index)
    if not 1 <= num <= 3:
        raise ValueError("positions must have one to three axes")
    if axes is not None:
        try:
            axes = axes if isinstance(axes, bytes) else bytes(list(axes))   # of a number, bytes() would make zeros
        except (TypeError, ValueError):
            axes = b""
        if len(axes) != half or max(axes) >= num:
            raise ValueError("pair_axes must hold an axis of positions for each of the table's pairs")
    return _Positions(positions.data_ptr(), positions.stride(0) if len(shape) == 3 else 0,
                      positions.stride(-2) if shape[-2] > 1 else 0, num, axes)


def kv_append_positioned(cache: PagedKVCache, block_table: torch.Tensor, seq_lens: torch.Tensor, k_new: torch.Tensor,
                         v_new: torch.Tensor, table: torch.Tensor, positions: torch.Tensor, q: Optional[torch.Tensor] = None,
                         q_out: Optional[torch.Tensor] = None, append_lens: Optional[torch.Tensor] = None,
                         pair_axes: Optional[Sequence[int]] = None, interleaved: bool = False,
                         status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """kv_append_rotated with the positions of the new tokens given, int32 [B, T] or [axes, B, T] (B or 1, up to
    three axes): a tree's tokens turn by their depth behind the context, image tokens by their time, height and
    width.  pair_axes: the axis of each of the table's channel pairs (None: the first); see pair_sections.  The
    tokens still go to the slots after seq_lens.  Tokens with a position that the table has not are skipped (status
    0x40): call again, from the same seq_lens, before their slots count as filled."""
    index = cache.device_index
    if index >= 0 and _get_device() != index:
        with torch.cuda.device(index):
            return kv_append_positioned(cache, block_table, seq_lens, k_new, v_new, table, positions, q, q_out, append_lens,
                                        pair_axes, interleaved, status, stream)
    return _append_rotated(cache, block_table, seq_lens, k_new, v_new, table, q, q_out, append_lens, interleaved,
                           (positions, pair_axes), status, stream)


def pair_sections(sections: Sequence[int]) -> bytes:
    """pair_axes of channel pairs in one span per axis, of these numbers of pairs."""
    return bytes(axis for axis, n in enumerate(sections) for _ in range(n))


def kv_keep_tokens(cache: PagedKVCache, block_table: torch.Tensor, seq_lens: torch.Tensor, starts: torch.Tensor,
                   keep: torch.Tensor, keep_lens: Optional[torch.Tensor] = None, lens_out: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Of the tokens from starts[b] on, keep[b, :keep_lens[b]] (default: all of keep [B, M], ascending, counted from
    the start) stay and move together behind the start; the others are given up.  Boxes and E4M3 scales follow.
    Returns the new lengths [B] (lens_out, allocated on the call's stream where not given)."""
    index = cache.device_index
    if index >= 0 and _get_device() != index:
        with torch.cuda.device(index):
            return kv_keep_tokens(cache, block_table, seq_lens, starts, keep, keep_lens, lens_out, status, stream)
    if block_table.dim() != 2 or keep.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages_per_seq] and keep [batch, tokens]")
    B, M = keep.shape
    maxp = block_table.shape[1]
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    if lens_out is None:
        with _allocating_on(stream):
            lens_out = torch.empty(B, dtype=torch.int32, device=cache.k_pool.device)
    code = _lib.qasa_kv_keep_tokens(
        cache.c_ref, _arg(block_table, "block_table", torch.int32, (B, maxp), index), maxp,
        _arg(seq_lens, "seq_lens", torch.int32, (B,), index), _arg(starts, "starts", torch.int32, (B,), index),
        _arg(keep, "keep", torch.int32, (B, M), index), M, _arg(keep_lens, "keep_lens", torch.int32, (B,), index),
        _arg(lens_out, "lens_out", torch.int32, (B,), index), B, _status_arg(status, index), _call_stream(stream, index))
    if code:
        _check(code, "qasa_kv_keep_tokens")
    return lens_out


def kv_copy_pages(cache: PagedKVCache, src_pages: torch.Tensor, dst_pages: torch.Tensor,
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Physical pages src_pages [n] become those of dst_pages [n]: K, V, boxes and scales."""
    index = cache.device_index
    if index >= 0 and _get_device() != index:
        with torch.cuda.device(index):
            return kv_copy_pages(cache, src_pages, dst_pages, status, stream)
    if src_pages.dim() != 1:
        raise ValueError("src_pages must be [pairs]")
    n = src_pages.shape[0]
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    code = _lib.qasa_kv_copy_pages(cache.c_ref, _arg(src_pages, "src_pages", torch.int32, (n,), index),
                                   _arg(dst_pages, "dst_pages", torch.int32, (n,), index), n, _status_arg(status, index),
                                   _call_stream(stream, index))
    if code:
        _check(code, "qasa_kv_copy_pages")


def kv_fork(cache: PagedKVCache, block_table: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor,
            new_pages: torch.Tensor, table_out: Optional[torch.Tensor] = None, lens_out: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Children go on from sequences parents [C]: (table_out [C, max_pages_per_seq], lens_out [C]).  Full pages are
    shared; a part-filled one is copied into new_pages[c], or taken over where that is negative.  Entries of table_out
    behind a child's pages are left as they were (-1 where it is allocated here, on the call's stream)."""
    index = cache.device_index
    if index >= 0 and _get_device() != index:
        with torch.cuda.device(index):
            return kv_fork(cache, block_table, seq_lens, parents, new_pages, table_out, lens_out, status, stream)
    if block_table.dim() != 2 or parents.dim() != 1:
        raise ValueError("block_table must be [batch, max_pages_per_seq] and parents [children]")
    (B, maxp), C = block_table.shape, parents.shape[0]
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    if table_out is None or lens_out is None:
        with _allocating_on(stream):
            if table_out is None:
                table_out = torch.full((C, maxp), -1, dtype=torch.int32, device=cache.k_pool.device)
            if lens_out is None:
                lens_out = torch.zeros(C, dtype=torch.int32, device=cache.k_pool.device)
    code = _lib.qasa_kv_fork(
        cache.c_ref, _arg(block_table, "block_table", torch.int32, (B, maxp), index), maxp,
        _arg(seq_lens, "seq_lens", torch.int32, (B,), index), B, _arg(parents, "parents", torch.int32, (C,), index),
        _arg(new_pages, "new_pages", torch.int32, (C,), index), C, _arg(table_out, "table_out", torch.int32, (C, maxp), index),
        _arg(lens_out, "lens_out", torch.int32, (C,), index), _status_arg(status, index), _call_stream(stream, index))
    if code:
        _check(code, "qasa_kv_fork")
    return table_out, lens_out


NO_WINDOW = 0x7FFFFFFF      # a window that every token is in


def _tokens(n: Optional[int]) -> int:
    """A count of tokens as the library takes it (None: all)."""
    return NO_WINDOW if n is None else min(int(n), NO_WINDOW)


def alloc_window_workspace(cache: PagedKVCache, batch: int, num_q_heads: int, max_q_tokens: int,
                           max_pages_per_seq: int, window: Optional[int] = None, sink_tokens: int = 0) -> torch.Tensor:
    """Workspace of window_attention calls of up to this batch, these tokens, pages, window and sinks."""
    n = int(_lib.qasa_window_workspace_size(batch, num_q_heads, cache.c_ref, max_q_tokens, max_pages_per_seq,
                                            _tokens(window), _tokens(sink_tokens)))
    return torch.empty(max(n, 16), dtype=torch.uint8, device=cache.k_pool.device)


def window_attention(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                     window: Optional[int] = None, sink_tokens: int = 0, q_lens: Optional[torch.Tensor] = None,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Attention of the newest tokens of every sequence: q [B, T, Hq, d] (or [B, Hq, d], one token each)
    holds the queries of the last q_lens[b] (default T) of its seq_lens[b] tokens, each of which sees
    itself and what came before within `window` tokens (None: everything) and the first `sink_tokens`.
    Rows at or past q_lens[b] of `out` are left as they were (unset where it is allocated here, on the call's
    stream)."""
    index = cache.device_index
    if index >= 0 and _get_device() != index:
        with torch.cuda.device(index):
            return window_attention(cache, q, block_table, seq_lens, window, sink_tokens, q_lens, scale, out, workspace,
                                    status, stream)
    value, shape = cache.value_dtype, q.shape
    if len(shape) == 4:
        B, T, hq, d = shape
    elif len(shape) == 3:
        (B, hq, d), T = shape, 1
    else:
        raise ValueError("q must be [batch, tokens, heads, head_dim] or [batch, heads, head_dim]")
    if d != cache.head_dim:
        raise ValueError("q must have the cache's head_dim")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages_per_seq]")
    maxp = block_table.shape[1]
    qp = _arg(q, "q", value, shape, index)
    if out is None or workspace is None:
        with _allocating_on(stream):
            if out is None:
                out = torch.empty_like(q)
            if workspace is None:
                workspace = alloc_window_workspace(cache, B, hq, T, maxp, window, sink_tokens)
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous memory on cuda:%d" % index)
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    code = _lib.qasa_window_attention(
        cache.c_ref, qp, hq, T, _arg(q_lens, "q_lens", torch.int32, (B,), index),
        _arg(block_table, "block_table", torch.int32, (B, maxp), index), maxp,
        _arg(seq_lens, "seq_lens", torch.int32, (B,), index), _tokens(window), _tokens(sink_tokens),
        scale or 0.0, _arg(out, "out", value, shape, index), workspace.data_ptr(), workspace.nbytes, B,
        _status_arg(status, index), _call_stream(stream, index))
    if code:
        _check(code, "qasa_window_attention")
    return out


def tree_masks(parents: torch.Tensor, lens: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
               depths: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Mask rows [B, T, ceil(T / 32)] and depths [B, T] (int32) of trees of drafted tokens given by parents [B, T]
    (an earlier token, or -1: the context).  Rows at or past lens[b] (default T) are left as they were (0 where they
    are allocated here, on the call's stream)."""
    index = parents.get_device()
    if index < 0:
        raise ValueError("parents must be on a CUDA device")
    if _get_device() != index:
        with torch.cuda.device(index):
            return tree_masks(parents, lens, mask, depths, status, stream)
    if parents.dim() != 2:
        raise ValueError("parents must be [batch, tokens]")
    B, T = parents.shape
    W = -(-T // 32)
    if mask is None or depths is None:
        with _allocating_on(stream):
            if mask is None:
                mask = torch.zeros((B, T, W), dtype=torch.int32, device=parents.device)
            if depths is None:
                depths = torch.zeros((B, T), dtype=torch.int32, device=parents.device)
    code = _lib.qasa_tree_masks(
        _arg(parents, "parents", torch.int32, (B, T), index), B, T, _arg(lens, "lens", torch.int32, (B,), index),
        _arg(mask, "mask", torch.int32, (B, T, W), index), _arg(depths, "depths", torch.int32, (B, T), index),
        _status_arg(status, index), _call_stream(stream, index))
    if code:
        _check(code, "qasa_tree_masks")
    return mask, depths


def alloc_tree_workspace(cache: PagedKVCache, batch: int, num_q_heads: int, max_q_tokens: int,
                         max_pages_per_seq: int) -> torch.Tensor:
    """Workspace of tree_attention calls of up to this batch, these tokens and pages."""
    n = int(_lib.qasa_tree_workspace_size(batch, num_q_heads, cache.c_ref, max_q_tokens, max_pages_per_seq))
    return torch.empty(max(n, 16), dtype=torch.uint8, device=cache.k_pool.device)


def tree_attention(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                   mask: torch.Tensor, q_lens: Optional[torch.Tensor] = None, window: Optional[int] = None,
                   sink_tokens: int = 0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Attention of a tree of drafted tokens: q [B, T, Hq, d] holds the queries of the last q_lens[b] (default T) of
    seq_lens[b] tokens.  Query t sees the drafted tokens of its row of mask (int32 words [B or 1, T, ceil(T / 32)], as
    tree_masks makes them) and of the context before them its window (None: everything) and the first sink_tokens.
    Rows at or past q_lens[b] of `out` are left as they were (unset where it is allocated here, on the call's
    stream)."""
    index = cache.device_index
    if index >= 0 and _get_device() != index:
        with torch.cuda.device(index):
            return tree_attention(cache, q, block_table, seq_lens, mask, q_lens, window, sink_tokens, scale, out, workspace,
                                  status, stream)
    shape = q.shape
    if len(shape) != 4 or block_table.dim() != 2:
        raise ValueError("q must be [batch, tokens, heads, head_dim] and block_table [batch, max_pages_per_seq]")
    B, T, hq, d = shape
    if d != cache.head_dim:
        raise ValueError("q must have the cache's head_dim")
    value, maxp, W = cache.value_dtype, block_table.shape[1], -(-T // 32)
    if mask.dim() != 3 or mask.shape[0] not in (1, B):
        raise ValueError("mask must be [batch or 1, tokens, words]")
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    qp = _arg(q, "q", value, shape, index)
    if out is None or workspace is None:
        with _allocating_on(stream):
            if out is None:
                out = torch.empty_like(q)
            if workspace is None:
                workspace = alloc_tree_workspace(cache, B, hq, T, maxp)
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous memory on cuda:%d" % index)
    code = _lib.qasa_tree_attention(
        cache.c_ref, qp, hq, T, _arg(q_lens, "q_lens", torch.int32, (B,), index),
        _arg(mask, "mask", torch.int32, (mask.shape[0], T, W), index), T * W if mask.shape[0] > 1 else 0,
        _arg(block_table, "block_table", torch.int32, (B, maxp), index), maxp,
        _arg(seq_lens, "seq_lens", torch.int32, (B,), index), _tokens(window), _tokens(sink_tokens), scale or 0.0,
        _arg(out, "out", value, shape, index), workspace.data_ptr(), workspace.nbytes, B, _status_arg(status, index),
        _call_stream(stream, index))
    if code:
        _check(code, "qasa_tree_attention")
    return out


def rebuild_page_bounds(cache: PagedKVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                        status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Recompute every page box of the batch from the keys in the pool."""
    B = int(seq_lens.shape[0])
    code = _lib.qasa_rebuild_page_bounds(cache.c_ref, _ptr(_contig(block_table, "block_table")),
                                         int(block_table.shape[1]), _ptr(_contig(seq_lens, "seq_lens")), B,
                                         _ptr(status), _stream(stream))
    _check(code, "qasa_rebuild_page_bounds")


def budget_pages(budget: Union[int, float, torch.Tensor], seq_lens: torch.Tensor,
                 page_size: int) -> torch.Tensor:
    """Per-sequence page budget as an int32 device tensor.

    int: that many pages for every sequence.  float in (0, 1]: ceil(fraction *
    N_b) pages (needs the lengths on the host, so a device ``seq_lens`` is
    copied back).  Tensor: used as is.
    """
    if isinstance(budget, torch.Tensor):
        return budget.to(device=seq_lens.device, dtype=torch.int32).contiguous()
    if isinstance(budget, float):
        lens = seq_lens.detach().to("cpu", torch.int64).tolist()
        k = [max(1, math.ceil(budget * ((L + page_size - 1) // page_size) - 1e-9)) for L in lens]
        return torch.tensor(k, dtype=torch.int32, device=seq_lens.device)
    return torch.full((int(seq_lens.shape[0]),), int(budget), dtype=torch.int32,
                      device=seq_lens.device)


def select_pages(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, budget, max_budget: int,
                 selected: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    B, Hq = int(q.shape[0]), int(q.shape[1])
    with _allocating_on(stream):
        bud = budget_pages(budget, seq_lens, cache.page_size)
        if selected is None:
            selected = torch.empty((B, cache.num_kv_heads, max_budget), dtype=torch.int32,
                                   device=q.device)
        if workspace is None:
            workspace = alloc_workspace(cache, B, Hq, int(block_table.shape[1]))
    code = _lib.qasa_select_pages(cache.c_ref, _ptr(_contig(q, "q")), Hq, _ptr(block_table),
                                  int(block_table.shape[1]), _ptr(seq_lens), _ptr(bud), max_budget,
                                  _ptr(selected), _ptr(scores), _ptr(workspace),
                                  workspace.numel(), B, _ptr(status), _stream(stream))
    _check(code, "qasa_select_pages")
    return selected


def sparse_attention(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor,
                     seq_lens: torch.Tensor, budget, selected: torch.Tensor,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    B, Hq = int(q.shape[0]), int(q.shape[1])
    with _allocating_on(stream):
        bud = budget_pages(budget, seq_lens, cache.page_size)
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            workspace = alloc_workspace(cache, B, Hq, int(block_table.shape[1]))
    code = _lib.qasa_sparse_attention(cache.c_ref, _ptr(_contig(q, "q")), Hq, _ptr(block_table),
                                      int(block_table.shape[1]), _ptr(seq_lens), _ptr(bud),
                                      int(selected.shape[-1]), _ptr(selected),
                                      float(scale or 0.0), _ptr(out), _ptr(workspace),
                                      workspace.numel(), B, _ptr(status), _stream(stream))
    _check(code, "qasa_sparse_attention")
    return out


def sparse_decode_attention(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor,
                            seq_lens: torch.Tensor, budget, max_budget: Optional[int] = None,
                            scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                            selected: Optional[torch.Tensor] = None,
                            scores: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            status: Optional[torch.Tensor] = None,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One decode step: (out [B, Hq, d], selected [B, Hkv, max_budget] ascending, -1 padded)."""
    B, Hq = int(q.shape[0]), int(q.shape[1])
    maxp = int(block_table.shape[1])
    if max_budget is None:
        max_budget = selected.shape[-1] if selected is not None else max(2, maxp)
    with _allocating_on(stream):
        bud = budget_pages(budget, seq_lens, cache.page_size)
        if out is None:
            out = torch.empty_like(q)
        if selected is None:
            selected = torch.empty((B, cache.num_kv_heads, max_budget), dtype=torch.int32,
                                   device=q.device)
        if workspace is None:
            workspace = alloc_workspace(cache, B, Hq, maxp)
    code = _lib.qasa_sparse_decode_attention(cache.c_ref, _ptr(_contig(q, "q")), Hq,
                                             _ptr(block_table), maxp, _ptr(seq_lens), _ptr(bud),
                                             int(max_budget), float(scale or 0.0), _ptr(out),
                                             _ptr(selected), _ptr(scores), _ptr(workspace),
                                             workspace.numel(), B, _ptr(status), _stream(stream))
    _check(code, "qasa_sparse_decode_attention")
    return out, selected


def sparse_decode_attention_noalloc(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor,
                                    seq_lens: torch.Tensor, budget, max_budget: int,
                                    out: torch.Tensor, selected: torch.Tensor,
                                    scale: Optional[float] = None,
                                    scores: Optional[torch.Tensor] = None,
                                    status: Optional[torch.Tensor] = None, stream=None) -> int:
    """The decode step without a workspace, for callers that cannot allocate
    device memory: the library's fixed device buffer serves as scratch (see
    qasa.h).  The caller passes every input and output; returns the status code
    (QASA_ERR_WORKSPACE when the shape needs more scratch than the buffer)."""
    B, Hq = int(q.shape[0]), int(q.shape[1])
    with _allocating_on(stream):
        bud = budget if isinstance(budget, torch.Tensor) else budget_pages(budget, seq_lens, cache.page_size)
    return int(_lib.qasa_sparse_decode_attention_noalloc(
        cache.c_ref, _ptr(_contig(q, "q")), Hq, _ptr(block_table), int(block_table.shape[1]),
        _ptr(seq_lens), _ptr(bud), int(max_budget), float(scale or 0.0), _ptr(out), _ptr(selected),
        _ptr(scores), B, _ptr(status), _stream(stream)))


def alloc_host_workspace(cache: PagedKVCache, batch: int, num_q_heads: int, max_pages_per_seq: int,
                         max_budget: int, device=None) -> torch.Tensor:
    n = int(_lib.qasa_host_decode_workspace_size(batch, num_q_heads, cache.c_ref, max_pages_per_seq, max_budget))
    if batch and not n:
        raise QasaError("unsupported shape for the host-buffer decode step")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or cache.k_pool.device)


def sparse_decode_attention_host(cache: PagedKVCache, q_host: torch.Tensor, block_table_host: torch.Tensor,
                                 seq_lens_host: torch.Tensor, budget_host: torch.Tensor, max_budget: int,
                                 out_host: torch.Tensor, selected_host: torch.Tensor,
                                 workspace: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                                 status: Optional[torch.Tensor] = None, stream=None) -> int:
    """The decode step with host (preferably pinned) inputs and outputs: the
    kernels access pinned buffers in place where the device can address them,
    else the copies and kernels are enqueued on the stream (synchronise before
    reading either way)."""
    B, Hq = int(q_host.shape[0]), int(q_host.shape[1])
    maxp = int(block_table_host.shape[1])
    if workspace is None:
        with _allocating_on(stream):
            workspace = alloc_host_workspace(cache, B, Hq, maxp, max_budget)
    code = _lib.qasa_sparse_decode_attention_host(
        cache.c_ref, _ptr(_contig(q_host, "q_host")), Hq, _ptr(_contig(block_table_host, "block_table_host")), maxp,
        _ptr(_contig(seq_lens_host, "seq_lens_host")), _ptr(_contig(budget_host, "budget_host")), int(max_budget),
        float(scale or 0.0), _ptr(_contig(out_host, "out_host")), _ptr(_contig(selected_host, "selected_host")),
        _ptr(workspace), workspace.numel(), B, _ptr(status), _stream(stream))
    _check(code, "qasa_sparse_decode_attention_host")
    return code


def host_call_is_direct(q_host: torch.Tensor, block_table_host: torch.Tensor, seq_lens_host: torch.Tensor,
                        budget_host: torch.Tensor, out_host: torch.Tensor, selected_host: torch.Tensor) -> bool:
    """True when sparse_decode_attention_host with these buffers lets the
    kernels read and write them in host memory (no copies launched)."""
    return bool(_lib.qasa_host_call_is_direct(*(_ptr(t) for t in (q_host, block_table_host, seq_lens_host,
                                                                  budget_host, out_host, selected_host))))


def dense_decode_attention(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor,
                           seq_lens: torch.Tensor, scale: Optional[float] = None,
                           out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    B, Hq = int(q.shape[0]), int(q.shape[1])
    maxp = int(block_table.shape[1])
    with _allocating_on(stream):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            workspace = alloc_workspace(cache, B, Hq, maxp)
    code = _lib.qasa_dense_decode_attention(cache.c_ref, _ptr(_contig(q, "q")), Hq,
                                            _ptr(block_table), maxp, _ptr(seq_lens),
                                            float(scale or 0.0), _ptr(out), _ptr(workspace),
                                            workspace.numel(), B, _ptr(status), _stream(stream))
    _check(code, "qasa_dense_decode_attention")
    return out


def page_attention_mass(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, scale: Optional[float] = None,
                        mass: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Share of the dense attention of each (sequence, KV head) on each page,
    [batch, num_kv_heads, max_pages_per_seq] float32 (pages >= N_b: zero when
    ``mass`` is allocated here, untouched otherwise)."""
    B, Hq = int(q.shape[0]), int(q.shape[1])
    maxp = int(block_table.shape[1])
    if mass is None:
        with _allocating_on(stream):
            mass = torch.zeros((B, cache.num_kv_heads, maxp), dtype=torch.float32, device=q.device)
    code = _lib.qasa_page_attention_mass(cache.c_ref, _ptr(_contig(q, "q")), Hq, _ptr(block_table), maxp,
                                         _ptr(seq_lens), float(scale or 0.0), _ptr(_contig(mass, "mass")),
                                         B, _ptr(status), _stream(stream))
    _check(code, "qasa_page_attention_mass")
    return mass


def page_hit_rate(cache: PagedKVCache, mass: torch.Tensor, seq_lens: torch.Tensor,
                  budget_pages: torch.Tensor, selected: torch.Tensor,
                  status: Optional[torch.Tensor] = None, stream=None):
    """(hits int32, covered float32, best float32), each [batch, num_kv_heads]:
    how many selected pages are among the k_b pages of largest mass, the mass
    the selection covers and the largest mass any k_b pages cover."""
    B, Hkv, maxp = (int(x) for x in mass.shape)
    mb = int(selected.shape[2])
    with _allocating_on(stream):
        hits = torch.empty((B, Hkv), dtype=torch.int32, device=mass.device)
        covered = torch.empty((B, Hkv), dtype=torch.float32, device=mass.device)
        best = torch.empty((B, Hkv), dtype=torch.float32, device=mass.device)
    code = _lib.qasa_page_hit_rate(cache.c_ref, _ptr(_contig(mass, "mass")), maxp, _ptr(seq_lens),
                                   _ptr(budget_pages), mb, _ptr(_contig(selected, "selected")), B,
                                   _ptr(hits), _ptr(covered), _ptr(best), _ptr(status), _stream(stream))
    _check(code, "qasa_page_hit_rate")
    return hits, covered, best


def decode_device_errors(code: int) -> Sequence[str]:
    return [msg for bit, msg in DEVERR.items() if code & bit]
