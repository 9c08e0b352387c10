"""split_kv_decode_distattention_gb300: split-KV decode attention over a paged KV cache.

This module is a thin Python binding of libdattn.so, the C-ABI library built from ``csrc/``.
It only marshals arguments: torch tensors become device pointers, and the current torch
stream becomes the launch stream. Every step of the computation runs in the library's
CUDA kernels. There is no CPU fallback: if the library is missing, the first call raises.

Entry points, with the same names as in include/dattn.h:
  dattn_kv_append    paged KV append (bf16, or 8-bit E4M3 or 4-bit codes with row scales),
                     plus logical-page k_max/k_min statistics
  dattn_partial      MicroAttention partials (m, e, MA) over explicit chunks of pages
  dattn_merge        log-sum-exp aggregation of partials
  dattn_decode       fused split-KV decode, dense or block-sparse
  dattn_append_decode one decode step with its one-token append, in one launch
  dattn_decode_multi fused decode of T new query tokens per request, causal over them
  dattn_page_select  page scoring and top-K selection for retrieval heads
  dattn_prefill      block-sparse prefill of a chunk of new tokens (64-token key blocks)
  dattn_rope         rotary positions of queries or keys, and their gradient
  dattn_rope_append  the append with the rotation of queries and keys applied on the way
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = [
    "KVLayout", "SparseConfig", "DattnError", "load_library", "library_path",
    "dattn_kv_append", "dattn_partial", "dattn_merge", "dattn_decode", "dattn_page_select",
    "dattn_append_decode", "dattn_merge_gathered", "dattn_rope", "dattn_rope_append",
    "dattn_rope_frequencies", "Rotation",
    "dattn_decode_noalloc", "dattn_decode_multi", "dattn_prefill", "PrefillSparseConfig",
    "dattn_workspace_size", "dattn_workspace_init", "dattn_auto_splits", "dattn_split_range",
    "dattn_split_owner", "dattn_status_string", "dattn_version", "Workspace",
    "HEAD_DENSE", "HEAD_RETRIEVAL", "HEAD_STREAMING", "DEVERR", "KV_BF16", "KV_FP8_E4M3",
    "KV_INT4", "KV_MIXED", "KV_FP8_BLOCK", "mixed_pool_bytes", "kv_scale_floats",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdattn.so")
_lib = None
_lock = threading.Lock()

HEAD_DENSE, HEAD_RETRIEVAL, HEAD_STREAMING = 0, 1, 2
KV_BF16, KV_FP8_E4M3, KV_INT4, KV_MIXED = 0, 1, 2, 3
KV_FP8_BLOCK = 5
_QUANT = (KV_FP8_E4M3, KV_INT4, KV_MIXED, KV_FP8_BLOCK)
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by-parts": 3}
DEVERR = {"UNMAPPED_PAGE": 0x1, "PAGE_OOB": 0x2, "LEN_OOB": 0x4, "TIMEOUT": 0x8,
          "CHUNK_OOB": 0x10, "SELECT_OOB": 0x20, "SMEM_ALIGN": 0x40}


class DattnError(RuntimeError):
    """A dattn call returned a status other than DATTN_OK."""


class _Layout(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("max_pages_per_req", ctypes.c_int32),
                ("kv_format", ctypes.c_int32), ("kv_scale", ctypes.c_void_p),
                ("head_format", ctypes.c_void_p)]


class _Sparse(ctypes.Structure):
    _fields_ = [("head_kind", ctypes.c_void_p), ("sinks", ctypes.c_int32),
                ("local", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("selected", ctypes.c_void_p), ("selected_phys", ctypes.c_void_p)]


class _PrefillSparse(ctypes.Structure):
    _fields_ = [("head_kind", ctypes.c_void_p), ("sink_blocks", ctypes.c_int32),
                ("local_blocks", ctypes.c_int32), ("max_sel", ctypes.c_int32),
                ("qblock_stride", ctypes.c_int32), ("block_lists", ctypes.c_void_p)]


class _Rotation(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("amplitude", ctypes.c_float), ("turns", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I = ctypes.c_int32
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_SIGS = {
    "dattn_kv_append": (_I, [ctypes.POINTER(_Layout), _P, _P, _P, _P, _P, _I, _I, _P, _P, _P]),
    "dattn_partial": (_I, [ctypes.POINTER(_Layout), _P, _P, _P, _I, _I, _F, _P, _I, _P, _P, _P,
                           _P, _P, _P, _P, _SZ, _I, _P, _P]),
    "dattn_merge": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "dattn_merge_gathered": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "dattn_decode": (_I, [ctypes.POINTER(_Layout), _P, _P, _P, _I, _I, _F, _P,
                          ctypes.POINTER(_Sparse), _I, _P, _SZ, _P, _P, _P, _P, _P]),
    "dattn_page_select": (_I, [ctypes.POINTER(_Layout), _P, _P, _I, _I, _P, _P, _I, _P, _P, _P,
                               _SZ, _I, _P, _P]),
    "dattn_append_decode": (_I, [ctypes.POINTER(_Layout), _P, _P, _P, _P, _P, _P, _I, _I, _F, _P,
                                 ctypes.POINTER(_Sparse), _I, _P, _SZ, _P, _P, _P, _P, _P]),
    "dattn_decode_noalloc": (_I, [ctypes.POINTER(_Layout), _P, _P, _P, _I, _I, _F, _P,
                                  ctypes.POINTER(_Sparse), _I, _P, _P, _P, _P, _P]),
    "dattn_decode_multi": (_I, [ctypes.POINTER(_Layout), _P, _P, _P, _I, _I, _I, _F, _P, _I, _P,
                                _SZ, _P, _P, _P, _P, _P]),
    "dattn_prefill": (_I, [ctypes.POINTER(_Layout), _P, _P, _P, _I, _I, _I, _F, _P,
                           ctypes.POINTER(_PrefillSparse), _P, _P, _P, _P, _P]),
    "dattn_rope_frequencies": (_I, [_I, _F, _I, _F, _F, _F, _F, _P]),
    "dattn_rope_turns": (_I, [_I, _P, _P]),
    "dattn_rope": (_I, [ctypes.POINTER(_Rotation), _P, _I64, _P, _I64, _I, _I, _I, _I, _P, _I,
                        _P]),
    "dattn_rope_append": (_I, [ctypes.POINTER(_Layout), _P, _P, _P, ctypes.POINTER(_Rotation),
                               _P, _I64, _P, _I64, _P, _I64, _I, _I, _I, _P, _P, _P, _P, _I, _P,
                               _P]),
    "dattn_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "dattn_workspace_init": (_I, [_P, _SZ, _P]),
    "dattn_auto_splits": (_I, [_I64]),
    "dattn_split_range": (None, [_I64, _I, _I, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "dattn_split_owner": (_I, [_I64, _I64, _I]),
    "dattn_status_string": (ctypes.c_char_p, [_I]),
    "dattn_version": (ctypes.c_char_p, []),
}


def library_path() -> str:
    return _LIB_PATH


def load_library(path: str | None = None):
    """Load libdattn.so (built in-tree by ``_build.build()``); raise if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _LIB_PATH
        if not os.path.exists(p):
            raise DattnError(
                f"{p} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(p)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def _check(status: int, what: str):
    if status != 0:
        msg = load_library().dattn_status_string(status).decode()
        raise DattnError(f"{what} failed: {msg}")


def _stream_on(stream, device):
    """The launch stream's handle: the given stream's, else the device's current one (by the raw
    getter: building a Stream object costs about as much as the launch)."""
    return stream.cuda_stream if stream is not None else \
        torch._C._cuda_getCurrentRawStream(device)


def _elsewhere(t, here):
    if t.get_device() < 0:
        raise ValueError("expected a CUDA tensor")
    raise ValueError(f"tensors of {t.device} and cuda:{here} in one call")


def _at(t, here):
    """The pointer of a contiguous tensor on device `here`."""
    if t is None:
        return None
    if t.get_device() != here:
        _elsewhere(t, here)
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _launch_device(t):
    """The device of t, which has to be the current one: the launch goes there."""
    here = t.get_device()
    if here < 0:
        raise ValueError("expected a CUDA tensor")
    if here != torch.cuda.current_device():
        raise ValueError(f"a tensor of {t.device} in a call on cuda:{torch.cuda.current_device()}")
    return here


def _layout_device(layout, t):
    """The device of a call over `layout`, t's: the current one, with the layout's tensors on it."""
    here = _launch_device(t)
    if layout.device != here:
        _elsewhere(layout.block_table, here)
    return here


def _bf16(t, name):
    if t is not None and t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    return t


def _i32(t, name):
    if t is not None and t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    return t


def _f32(t, name):
    if t is not None and t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    return t


def _size(t, n: int, name: str):
    """A tensor argument must hold at least the n elements the call will touch: the kernels
    see only a pointer, so a short tensor would be read or written past its end."""
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements; the call needs {n}")
    return t


def mixed_pool_bytes(num_pages: int, head_format, head_dim: int, page_size: int) -> int:
    """Bytes of one (K or V) mixed pool: the 8-bit region [num_pages][H8][P][d], then the 4-bit
    region [num_pages][H4][P][d/2]."""
    h4 = sum(1 for f in head_format if f == KV_INT4)
    h8 = len(head_format) - h4
    return num_pages * page_size * (h8 * head_dim + h4 * (head_dim // 2))


def kv_scale_floats(kv_format: int, num_pages: int, num_kv_heads: int, page_size: int) -> int:
    """Floats of kv_scale: two per row (the row-scaled formats), or two per 16-token block, padded
    to a multiple of four (KV_FP8_BLOCK); 0 for bf16."""
    n = num_pages * num_kv_heads * page_size
    if kv_format == KV_FP8_BLOCK:
        return -(-(n // 16) // 2) * 4
    return 2 * n if kv_format in _QUANT else 0


def _layout_sizes(layout, B: int, k_pool, v_pool, stats=None):
    """The pools, block table, scales and statistics must cover the layout for B requests."""
    pool, scales, stat, table = layout.sizes
    _size(k_pool, pool, "k_pool")
    _size(v_pool, pool, "v_pool")
    _size(layout.block_table, B * table, "block_table")
    if scales:
        _size(layout.kv_scale, scales, "kv_scale")
    _size(stats, stat, "stats")


def _pool(layout, t, name):
    """A K or V pool must hold the layout's element type: bf16, uint8 E4M3 codes, or uint8
    bytes of two 4-bit codes (the mixed pool: both kinds of bytes)."""
    if t is not None and t.dtype not in layout.pool_types:
        raise TypeError(f"{name} must be {layout.pool_types[0]} for this layout")
    return t


class KVLayout:
    """Shape of a paged pool [num_pages][Hkv][P][d] plus its int32 block table [B][max_pages].

    kv_format KV_BF16: the pools hold bf16 values. KV_FP8_E4M3: they hold uint8 E4M3 codes,
    and kv_scale (float32 [num_pages][Hkv][P/16][2][16]) holds one scale per row: for the 16
    tokens of each logical page, their K scales, then their V scales. KV_INT4: they hold
    [num_pages][Hkv][P][d/2] bytes of two 4-bit codes each (code + 8, even channel in the low
    nibble), with kv_scale as for KV_FP8_E4M3. KV_MIXED: head_format[h] (KV_FP8_E4M3 or
    KV_INT4) gives each KV head's format; the pools are that many bytes
    (mixed_pool_bytes): the 8-bit heads' region, then the 4-bit heads' region, each head at
    its index among the heads of its format. KV_FP8_BLOCK: uint8 E4M3 codes with one power-of-two
    K scale and V scale per logical page, kv_scale float32 [num_pages][Hkv][P/16][2] padded to
    kv_scale_floats(...) elements.
    """

    def __init__(self, num_pages: int, num_kv_heads: int, head_dim: int, page_size: int,
                 block_table: torch.Tensor, kv_format: int = KV_BF16,
                 kv_scale: torch.Tensor | None = None, head_format=None):
        _i32(block_table, "block_table")
        if kv_format in _QUANT:
            if kv_scale is None:
                raise ValueError("the quantized formats need kv_scale")
            _f32(kv_scale, "kv_scale")
        self.head_format = None
        self._head_format_c = None
        if kv_format == KV_MIXED:
            if head_format is None or len(head_format) != num_kv_heads:
                raise ValueError("the mixed format needs one head_format entry per KV head")
            self.head_format = [int(f) for f in head_format]
            self._head_format_c = (ctypes.c_int8 * num_kv_heads)(*self.head_format)
        self.block_table = block_table  # keeps the tensors alive
        self.kv_scale = kv_scale
        self.device = block_table.get_device()  # (-1: the host's, which no call takes)
        _at(block_table, self.device)
        if kv_format in _QUANT:
            _at(kv_scale, self.device)
        self.c = _Layout(num_pages, num_kv_heads, head_dim, page_size,
                         block_table.data_ptr(), block_table.shape[-1], kv_format,
                         kv_scale.data_ptr() if kv_scale is not None else None,
                         ctypes.addressof(self._head_format_c)
                         if self._head_format_c is not None else None)
        self.pool_types = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)) \
            if kv_format in _QUANT else (torch.bfloat16,)
        # elements of a pool, floats of kv_scale, elements of the statistics, block-table row width
        n = num_pages * num_kv_heads * page_size
        if kv_format == KV_MIXED:
            pool = mixed_pool_bytes(num_pages, self.head_format, head_dim, page_size)
        else:
            pool = n * (head_dim // 2 if kv_format == KV_INT4 else head_dim)
        self.sizes = (pool, kv_scale_floats(kv_format, num_pages, num_kv_heads, page_size),
                      n // 16 * 2 * head_dim, block_table.shape[-1])

    @property
    def kv_format(self): return self.c.kv_format

    @property
    def num_pages(self): return self.c.num_pages

    @property
    def num_kv_heads(self): return self.c.num_kv_heads

    @property
    def head_dim(self): return self.c.head_dim

    @property
    def page_size(self): return self.c.page_size


class SparseConfig:
    """Block-sparse settings: per-KV-head kinds, streaming window and retrieval selection."""

    def __init__(self, head_kind: torch.Tensor, sinks: int, local: int, top_k: int,
                 selected: torch.Tensor | None, selected_phys: torch.Tensor | None = None):
        if head_kind.dtype != torch.int8:
            raise TypeError("head_kind must be int8")
        for t, n in ((selected, "selected"), (selected_phys, "selected_phys")):
            if t is not None and (t.dtype != torch.int32 or not t.is_contiguous()):
                raise TypeError(f"{n} must be a contiguous int32 tensor")
        if selected is not None and selected_phys is not None and \
                selected_phys.numel() < selected.numel():
            raise ValueError("selected_phys must have the shape of selected")
        self.head_kind, self.selected, self.selected_phys = head_kind, selected, selected_phys
        self.c = _Sparse(head_kind.data_ptr(), sinks, local, top_k,
                         selected.data_ptr() if selected is not None else None,
                         selected_phys.data_ptr() if selected_phys is not None else None)


class PrefillSparseConfig:
    """Block-sparse prefill settings: per-KV-head kinds, the streaming heads' sink and local
    block counts, and the retrieval heads' key-block lists (int32 [B][Hkv][qblock_stride]
    [max_sel], row qb for query block qb, -1 padded)."""

    def __init__(self, head_kind: torch.Tensor, sink_blocks: int, local_blocks: int,
                 block_lists: torch.Tensor | None = None):
        if head_kind.dtype != torch.int8:
            raise TypeError("head_kind must be int8")
        _i32(block_lists, "block_lists")
        self.head_kind, self.block_lists = head_kind, block_lists
        qs, ms = (block_lists.shape[2], block_lists.shape[3]) if block_lists is not None else (0, 0)
        self.c = _PrefillSparse(head_kind.data_ptr(), sink_blocks, local_blocks, ms, qs,
                                block_lists.data_ptr() if block_lists is not None else None)


class Rotation:
    """Rotary positions of the first rot_dim channels (a multiple of 16): pairs (k, k + rot_dim/2),
    or (2k, 2k + 1) when interleaved, turned by position * f_k and scaled by amplitude.

    f_k comes from base and a scaling for long contexts: "none", "linear" (f_k / factor), "ntk"
    (the base raised) or "by-parts" (frequencies with fewer than `low` turns over original_len
    divided by factor, those with more than `high` kept, a ramp between); or is given as inv_freq,
    rot_dim / 2 numbers. base, factor and the other parameters are taken as fp32 numbers, inv_freq as
    fp64. The frequencies are kept as host data: a Rotation belongs to no device.
    """

    def __init__(self, rot_dim: int, interleaved: bool = False, base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, original_len: float = 8192.0,
                 low: float = 1.0, high: float = 4.0, amplitude: float = 1.0, inv_freq=None):
        n = rot_dim // 2
        if inv_freq is None:
            inv_freq = dattn_rope_frequencies(rot_dim, base, scaling, factor, original_len, low,
                                              high) if rot_dim else []
        elif len(inv_freq) != n:
            raise ValueError(f"inv_freq holds {len(inv_freq)} frequencies; rot_dim / 2 = {n}")
        self.inv_freq = [float(f) for f in inv_freq]
        self._turns = (ctypes.c_uint64 * max(n, 1))()
        _check(load_library().dattn_rope_turns(n, (ctypes.c_double * max(n, 1))(*self.inv_freq),
                                               self._turns), "dattn_rope_turns")
        self.c = _Rotation(rot_dim, int(bool(interleaved)), amplitude,
                           ctypes.addressof(self._turns))

    @property
    def rot_dim(self): return self.c.rot_dim


def dattn_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none",
                           factor: float = 1.0, original_len: float = 8192.0, low: float = 1.0,
                           high: float = 4.0) -> list:
    """The rot_dim / 2 inverse frequencies of a scaling ("none", "linear", "ntk", "by-parts")."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    out = (ctypes.c_double * max(rot_dim // 2, 1))()
    _check(load_library().dattn_rope_frequencies(rot_dim, base, _SCALINGS[scaling], factor,
                                                 original_len, low, high, out),
           "dattn_rope_frequencies")
    return list(out)[:rot_dim // 2]


class Workspace:
    """A zeroed device workspace sized by dattn_workspace_size (allocated by torch)."""

    def __init__(self, items: int, Hq: int, Hkv: int, head_dim: int, top_k: int = 0,
                 num_splits: int = 0, device=None):
        self.nbytes = dattn_workspace_size(items, Hq, Hkv, head_dim, top_k, num_splits)
        n = max(self.nbytes, 256)
        self.buffer = torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def dattn_workspace_size(items, Hq, Hkv, head_dim, top_k=0, num_splits=0) -> int:
    return int(load_library().dattn_workspace_size(items, Hq, Hkv, head_dim, top_k, num_splits))


def dattn_workspace_init(ws: Workspace, stream=None):
    if ws.buffer.get_device() < 0:
        raise ValueError("expected a CUDA tensor")
    _check(load_library().dattn_workspace_init(
        ws.buffer.data_ptr(), ws.buffer.numel(), _stream_on(stream, torch.cuda.current_device())),
        "dattn_workspace_init")


def dattn_auto_splits(total_tiles: int) -> int:
    """The automatic split of total_tiles 16-token tiles, 16 to a CTA at least. A launch with
    num_splits=0 may take more CTAs (KV_FP8_BLOCK: 4 tiles each); size its workspace with
    num_splits=0."""
    return int(load_library().dattn_auto_splits(total_tiles))


def dattn_split_range(total_tiles: int, num_splits: int, cta: int):
    b, e = ctypes.c_int64(), ctypes.c_int64()
    load_library().dattn_split_range(total_tiles, num_splits, cta, ctypes.byref(b),
                                     ctypes.byref(e))
    return b.value, e.value


def dattn_split_owner(tile: int, total_tiles: int, num_splits: int) -> int:
    return int(load_library().dattn_split_owner(tile, total_tiles, num_splits))


def dattn_status_string(status: int) -> str:
    return load_library().dattn_status_string(status).decode()


def dattn_version() -> str:
    return load_library().dattn_version().decode()


def dattn_kv_append(layout: KVLayout, k_pool, v_pool, stats, k_new, v_new, seq_lens,
                    dev_err=None, stream=None):
    """Append k_new/v_new ([B][T][Hkv][d] bf16) at seq_lens (int32 [B], advanced by T)."""
    _pool(layout, k_pool, "k_pool"); _pool(layout, v_pool, "v_pool"); _bf16(stats, "stats")
    _bf16(k_new, "k_new"); _bf16(v_new, "v_new"); _i32(seq_lens, "seq_lens")
    B, T = k_new.shape[0], k_new.shape[1]
    Hkv, d = layout.num_kv_heads, layout.head_dim
    _layout_sizes(layout, B, k_pool, v_pool, stats)
    _size(k_new, B * T * Hkv * d, "k_new"); _size(v_new, B * T * Hkv * d, "v_new")
    _size(seq_lens, B, "seq_lens")
    here = _layout_device(layout, k_pool)
    _check(load_library().dattn_kv_append(
        ctypes.byref(layout.c), _at(k_pool, here), _at(v_pool, here), _at(stats, here),
        _at(k_new, here), _at(v_new, here), B, T, _at(seq_lens, here), _at(dev_err, here),
        _stream_on(stream, here)), "dattn_kv_append")


def _tokens(t, name, here=None):
    """A [tokens...][H][d] tensor whose heads are packed and whose tokens are evenly spaced (a
    contiguous tensor or a slice of a fused projection), on device `here` where that is given:
    (pointer, elements between tokens)."""
    size, step = t.shape, t.stride()
    dims = len(size)
    if dims != 3 and dims != 4:
        raise ValueError(f"{name} must be [tokens][heads][d] or [B][T][heads][d]")
    H, d = size[-2], size[-1]
    if step[-1] != 1 or (H > 1 and step[-2] != d):
        raise ValueError(f"the heads of {name} must be packed")
    if dims == 3:
        many, stride = size[0] > 1, step[0]
    else:
        B, T = size[0], size[1]
        many, stride = B > 1 or T > 1, step[0] if T == 1 else step[1]
        if B > 1 and T > 1 and step[0] != T * stride:
            raise ValueError(f"the tokens of {name} must be evenly spaced")
    device = t.get_device()
    if device < 0 or (here is not None and device != here):
        _elsewhere(t, here)
    return t.data_ptr(), stride if many else H * d


def dattn_rope(rotation: Rotation, x, out, positions, inverse: bool = False, stream=None):
    """Rotate x, bf16 or float32 [N][H][d] or [B][T][H][d], into out (same shape and type; may be
    x) at the int32 positions, one per token. inverse=True negates the angles: the gradient."""
    dtype = x.dtype
    f32 = dtype == torch.float32
    if not (f32 or dtype == torch.bfloat16) or out.dtype != dtype:
        raise TypeError("x and out must both be bfloat16 or both float32")
    size = x.shape
    if out.shape != size:
        raise ValueError("out must have the shape of x")
    _i32(positions, "positions")
    here = x.get_device()
    xp, xs = _tokens(x, "x", here)
    op, os_ = _tokens(out, "out", here)
    H, d = size[-2], size[-1]
    N = size[0] if len(size) == 3 else size[0] * size[1]
    _size(positions, N, "positions")
    _launch_device(x)
    _check(load_library().dattn_rope(
        ctypes.byref(rotation.c), xp, xs, op, os_, N, H, d, f32, _at(positions, here),
        bool(inverse), _stream_on(stream, here)), "dattn_rope")


def dattn_rope_append(layout: KVLayout, k_pool, v_pool, stats, rotation: Rotation | None, q, k_new,
                      v_new, q_out, seq_lens, positions=None, new_lens=None, advance: bool = True,
                      dev_err=None, stream=None):
    """Rotate q ([B][T][Hq][d] bf16, into q_out, contiguous; both may be None) and k_new, and
    append the rotated keys and v_new ([B][T][Hkv][d] bf16) at seq_lens (int32 [B]), in one
    launch. q, k_new and v_new may be slices of a fused projection. positions (int32 [B][T])
    replaces seq_lens[b] + t as the rotation's positions; new_lens (int32 [B]) gives the new
    tokens of each request in a padded batch; advance=False leaves seq_lens as it is."""
    _pool(layout, k_pool, "k_pool"); _pool(layout, v_pool, "v_pool"); _bf16(stats, "stats")
    _bf16(q, "q"); _bf16(q_out, "q_out"); _bf16(k_new, "k_new"); _bf16(v_new, "v_new")
    _i32(seq_lens, "seq_lens"); _i32(positions, "positions"); _i32(new_lens, "new_lens")
    Hkv, d = layout.num_kv_heads, layout.head_dim
    size = k_new.shape
    if len(size) != 4 or size[2] != Hkv or size[3] != d or v_new.shape != size:
        raise ValueError("k_new and v_new must be bf16 [B][T][Hkv][d]")
    B, T = size[0], size[1]
    Hq, qp, qs = 0, None, 0
    if q is not None:
        qsize = q.shape
        if q_out is None:
            raise ValueError("q and q_out come together")
        if len(qsize) != 4 or qsize[0] != B or qsize[1] != T or qsize[3] != d or qsize[2] == 0:
            raise ValueError("q must be bf16 [B][T][Hq][d]")
        Hq = qsize[2]
        _size(q_out, B * T * Hq * d, "q_out")
    elif q_out is not None:
        raise ValueError("q and q_out come together")
    _layout_sizes(layout, B, k_pool, v_pool, stats)
    _size(seq_lens, B, "seq_lens"); _size(new_lens, B, "new_lens")
    _size(positions, B * T, "positions")
    here = _layout_device(layout, k_new)
    if q is not None:
        qp, qs = _tokens(q, "q", here)
    kp, ks = _tokens(k_new, "k_new", here)
    vp, vs = _tokens(v_new, "v_new", here)
    _check(load_library().dattn_rope_append(
        ctypes.byref(layout.c), _at(k_pool, here), _at(v_pool, here), _at(stats, here),
        ctypes.byref(rotation.c) if rotation is not None else None, qp, qs, kp, ks, vp, vs, B, T,
        Hq, _at(q_out, here), _at(seq_lens, here), _at(positions, here), _at(new_lens, here),
        bool(advance), _at(dev_err, here), _stream_on(stream, here)), "dattn_rope_append")


def dattn_partial(layout: KVLayout, k_pool, v_pool, q, scale: float, seq_lens, chunk_req,
                  chunk_page_indptr, chunk_pages, m, e, MA, ws: Workspace, num_splits=0,
                  dev_err=None, stream=None):
    """MicroAttention partials of C chunks: m, e fp32 [C][Hq], MA fp32 [C][Hq][d]."""
    _pool(layout, k_pool, "k_pool"); _pool(layout, v_pool, "v_pool"); _bf16(q, "q"); _i32(seq_lens, "seq_lens"); _i32(chunk_req, "chunk_req")
    _i32(chunk_page_indptr, "chunk_page_indptr"); _i32(chunk_pages, "chunk_pages")
    _f32(m, "m"); _f32(e, "e"); _f32(MA, "MA")
    B, Hq = q.shape[0], q.shape[1]
    C = chunk_req.shape[0]
    d = layout.head_dim
    _layout_sizes(layout, B, k_pool, v_pool)
    _size(q, B * Hq * d, "q"); _size(seq_lens, B, "seq_lens")
    _size(chunk_page_indptr, C + 1, "chunk_page_indptr")
    _size(m, C * Hq, "m"); _size(e, C * Hq, "e"); _size(MA, C * Hq * d, "MA")
    here = _layout_device(layout, k_pool)
    _check(load_library().dattn_partial(
        ctypes.byref(layout.c), _at(k_pool, here), _at(v_pool, here), _at(q, here), B, Hq, scale,
        _at(seq_lens, here), C, _at(chunk_req, here), _at(chunk_page_indptr, here),
        _at(chunk_pages, here), _at(m, here), _at(e, here), _at(MA, here), _at(ws.buffer, here),
        ws.buffer.numel(), num_splits, _at(dev_err, here), _stream_on(stream, here)),
        "dattn_partial")


def dattn_merge(chunk_indptr, m, e, MA, out=None, m_g=None, e_g=None, MA_g=None, dev_err=None,
                stream=None):
    """Aggregate partials per request (chunk ranges from chunk_indptr int32 [B+1])."""
    _i32(chunk_indptr, "chunk_indptr")
    for t, n in ((m, "m"), (e, "e"), (MA, "MA"), (out, "out"), (m_g, "m_g"), (e_g, "e_g"),
                 (MA_g, "MA_g")):
        _f32(t, n)
    B = chunk_indptr.shape[0] - 1
    C, Hq, d = MA.shape
    _size(m, C * Hq, "m"); _size(e, C * Hq, "e")
    _size(out, B * Hq * d, "out"); _size(m_g, B * Hq, "m_g"); _size(e_g, B * Hq, "e_g")
    _size(MA_g, B * Hq * d, "MA_g")
    here = _launch_device(MA)
    _check(load_library().dattn_merge(
        B, C, Hq, d, _at(chunk_indptr, here), _at(m, here), _at(e, here), _at(MA, here),
        _at(out, here), _at(m_g, here), _at(e_g, here), _at(MA_g, here), _at(dev_err, here),
        _stream_on(stream, here)), "dattn_merge")


def dattn_merge_gathered(m, e, MA, out=None, m_g=None, e_g=None, MA_g=None, dev_err=None,
                         stream=None):
    """Aggregate partials gathered from R ranks: m, e fp32 [R][B][Hq], MA fp32 [R][B][Hq][d]
    (rank r's dattn_partial over its pages, one chunk per request) -> out fp32 [B][Hq][d]."""
    for t, n in ((m, "m"), (e, "e"), (MA, "MA"), (out, "out"), (m_g, "m_g"), (e_g, "e_g"),
                 (MA_g, "MA_g")):
        _f32(t, n)
    if MA.dim() != 4:
        raise ValueError("MA must be fp32 [R][B][Hq][d]")
    R, B, Hq, d = MA.shape
    _size(m, R * B * Hq, "m"); _size(e, R * B * Hq, "e")
    _size(out, B * Hq * d, "out"); _size(m_g, B * Hq, "m_g"); _size(e_g, B * Hq, "e_g")
    _size(MA_g, B * Hq * d, "MA_g")
    here = _launch_device(MA)
    _check(load_library().dattn_merge_gathered(
        B, R, Hq, d, _at(m, here), _at(e, here), _at(MA, here), _at(out, here), _at(m_g, here),
        _at(e_g, here), _at(MA_g, here), _at(dev_err, here), _stream_on(stream, here)),
        "dattn_merge_gathered")


def _decode_sizes(layout, B, T, Hq, k_pool, v_pool, q, seq_lens, out, m_g, e_g, sparse):
    d, Hkv = layout.head_dim, layout.num_kv_heads
    _layout_sizes(layout, B, k_pool, v_pool)
    _size(q, B * T * Hq * d, "q"); _size(out, B * T * Hq * d, "out")
    _size(m_g, B * T * Hq, "m_g"); _size(e_g, B * T * Hq, "e_g"); _size(seq_lens, B, "seq_lens")
    if sparse is not None:
        _size(sparse.head_kind, Hkv, "head_kind")
        _size(sparse.selected, B * Hkv * sparse.c.top_k, "selected")


def dattn_decode(layout: KVLayout, k_pool, v_pool, q, scale: float, seq_lens, out,
                 ws: Workspace, m_g=None, e_g=None, sparse: SparseConfig | None = None,
                 num_splits=0, dev_err=None, stream=None):
    """Fused split-KV decode: out fp32 [B][Hq][d] (+ m_g, e_g fp32 [B][Hq])."""
    _pool(layout, k_pool, "k_pool"); _pool(layout, v_pool, "v_pool"); _bf16(q, "q"); _i32(seq_lens, "seq_lens"); _f32(out, "out")
    B, Hq = q.shape[0], q.shape[1]
    _decode_sizes(layout, B, 1, Hq, k_pool, v_pool, q, seq_lens, out, m_g, e_g, sparse)
    sp = ctypes.byref(sparse.c) if sparse is not None else None
    here = _layout_device(layout, k_pool)
    if sparse is not None:
        _at(sparse.head_kind, here); _at(sparse.selected, here); _at(sparse.selected_phys, here)
    _check(load_library().dattn_decode(
        ctypes.byref(layout.c), _at(k_pool, here), _at(v_pool, here), _at(q, here), B, Hq, scale,
        _at(seq_lens, here), sp, num_splits, _at(ws.buffer, here), ws.buffer.numel(),
        _at(out, here), _at(m_g, here), _at(e_g, here), _at(dev_err, here),
        _stream_on(stream, here)), "dattn_decode")


def dattn_append_decode(layout: KVLayout, k_pool, v_pool, stats, k_new, v_new, q, scale: float,
                        seq_lens, out, ws: Workspace, m_g=None, e_g=None,
                        sparse: SparseConfig | None = None, num_splits=0, dev_err=None,
                        stream=None):
    """dattn_kv_append of one token per request (k_new/v_new bf16 [B][1][Hkv][d]) and
    dattn_decode over the advanced lengths, in one launch (any pool format but KV_FP8_BLOCK; a
    quantized pool stores the new rows quantized as dattn_kv_append would): out fp32 [B][Hq][d]
    (+ m_g, e_g fp32 [B][Hq]); seq_lens advances by one."""
    _pool(layout, k_pool, "k_pool"); _pool(layout, v_pool, "v_pool"); _bf16(stats, "stats")
    _bf16(k_new, "k_new"); _bf16(v_new, "v_new"); _bf16(q, "q"); _i32(seq_lens, "seq_lens")
    _f32(out, "out")
    B, Hq = q.shape[0], q.shape[1]
    Hkv, d = layout.num_kv_heads, layout.head_dim
    if k_new.dim() != 4 or k_new.shape[1] != 1 or v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must be bf16 [B][1][Hkv][d]")
    _layout_sizes(layout, B, k_pool, v_pool, stats)
    _size(k_new, B * Hkv * d, "k_new"); _size(v_new, B * Hkv * d, "v_new")
    _decode_sizes(layout, B, 1, Hq, k_pool, v_pool, q, seq_lens, out, m_g, e_g, sparse)
    sp = ctypes.byref(sparse.c) if sparse is not None else None
    here = _layout_device(layout, k_pool)
    if sparse is not None:
        _at(sparse.head_kind, here); _at(sparse.selected, here); _at(sparse.selected_phys, here)
    _check(load_library().dattn_append_decode(
        ctypes.byref(layout.c), _at(k_pool, here), _at(v_pool, here), _at(stats, here),
        _at(k_new, here), _at(v_new, here), _at(q, here), B, Hq, scale, _at(seq_lens, here), sp,
        num_splits, _at(ws.buffer, here), ws.buffer.numel(), _at(out, here), _at(m_g, here),
        _at(e_g, here), _at(dev_err, here), _stream_on(stream, here)), "dattn_append_decode")


def dattn_decode_multi(layout: KVLayout, k_pool, v_pool, q, scale: float, seq_lens, out,
                       ws: Workspace, m_g=None, e_g=None, num_splits=0, dev_err=None, stream=None):
    """T query tokens per request (q bf16 [B][T][Hq][d]), causal over the T newest tokens:
    out fp32 [B][T][Hq][d] (+ m_g, e_g fp32 [B][T][Hq]). The workspace is sized for T * Hq
    query heads."""
    _pool(layout, k_pool, "k_pool"); _pool(layout, v_pool, "v_pool"); _bf16(q, "q")
    _i32(seq_lens, "seq_lens"); _f32(out, "out")
    B, T, Hq = q.shape[0], q.shape[1], q.shape[2]
    _decode_sizes(layout, B, T, Hq, k_pool, v_pool, q, seq_lens, out, m_g, e_g, None)
    here = _layout_device(layout, k_pool)
    _check(load_library().dattn_decode_multi(
        ctypes.byref(layout.c), _at(k_pool, here), _at(v_pool, here), _at(q, here), B, T, Hq,
        scale, _at(seq_lens, here), num_splits, _at(ws.buffer, here), ws.buffer.numel(),
        _at(out, here), _at(m_g, here), _at(e_g, here), _at(dev_err, here),
        _stream_on(stream, here)), "dattn_decode_multi")


def dattn_prefill(layout: KVLayout, k_pool, v_pool, q, scale: float, seq_lens, out, m=None,
                  e=None, sparse: PrefillSparseConfig | None = None, dev_err=None, stream=None):
    """Block-sparse (sparse given) or causal prefill of q bf16 [B][Tq][Hq][d], the last Tq
    tokens of each request: out fp32 [B][Tq][Hq][d] (+ m, e fp32 [B][Tq][Hq])."""
    _pool(layout, k_pool, "k_pool"); _pool(layout, v_pool, "v_pool"); _bf16(q, "q")
    _i32(seq_lens, "seq_lens"); _f32(out, "out"); _f32(m, "m"); _f32(e, "e")
    B, Tq, Hq = q.shape[0], q.shape[1], q.shape[2]
    _decode_sizes(layout, B, Tq, Hq, k_pool, v_pool, q, seq_lens, out, m, e, None)
    if sparse is not None:
        _size(sparse.head_kind, layout.num_kv_heads, "head_kind")
        if sparse.block_lists is not None and (sparse.block_lists.dim() != 4 or
                                               sparse.block_lists.shape[0] < B or
                                               sparse.block_lists.shape[1] < layout.num_kv_heads):
            raise ValueError("block_lists must be int32 [B][Hkv][qblock_stride][max_sel]")
    sp = ctypes.byref(sparse.c) if sparse is not None else None
    here = _layout_device(layout, k_pool)
    if sparse is not None:
        _at(sparse.head_kind, here); _at(sparse.block_lists, here)
    _check(load_library().dattn_prefill(
        ctypes.byref(layout.c), _at(k_pool, here), _at(v_pool, here), _at(q, here), B, Tq, Hq,
        scale, _at(seq_lens, here), sp, _at(out, here), _at(m, here), _at(e, here),
        _at(dev_err, here), _stream_on(stream, here)), "dattn_prefill")


def dattn_decode_noalloc(layout: KVLayout, k_pool, v_pool, q, scale: float, seq_lens, out,
                         m_g=None, e_g=None, sparse: SparseConfig | None = None, num_splits=0,
                         dev_err=None, stream=None):
    """dattn_decode with the library's fixed 8 MiB scratch array instead of a workspace.

    For callers that cannot allocate device memory. Calls on one device share the array, so
    they must not overlap on the GPU. The first call on a device should come before any
    stream capture.
    """
    _pool(layout, k_pool, "k_pool"); _pool(layout, v_pool, "v_pool"); _bf16(q, "q"); _i32(seq_lens, "seq_lens"); _f32(out, "out")
    B, Hq = q.shape[0], q.shape[1]
    _decode_sizes(layout, B, 1, Hq, k_pool, v_pool, q, seq_lens, out, m_g, e_g, sparse)
    sp = ctypes.byref(sparse.c) if sparse is not None else None
    here = _layout_device(layout, k_pool)
    if sparse is not None:
        _at(sparse.head_kind, here); _at(sparse.selected, here); _at(sparse.selected_phys, here)
    _check(load_library().dattn_decode_noalloc(
        ctypes.byref(layout.c), _at(k_pool, here), _at(v_pool, here), _at(q, here), B, Hq, scale,
        _at(seq_lens, here), sp, num_splits, _at(out, here), _at(m_g, here), _at(e_g, here),
        _at(dev_err, here), _stream_on(stream, here)), "dattn_decode_noalloc")


def dattn_page_select(layout: KVLayout, stats, q, seq_lens, head_kind, top_k: int, selected,
                      ws: Workspace, num_splits=0, dev_err=None, stream=None, selected_phys=None):
    """Top-K physical pages per retrieval head into selected int32 [B][Hkv][top_k] (and their
    pool pages into selected_phys, of the same shape, when given)."""
    _bf16(stats, "stats"); _bf16(q, "q"); _i32(seq_lens, "seq_lens"); _i32(selected, "selected")
    _i32(selected_phys, "selected_phys")
    B, Hq = q.shape[0], q.shape[1]
    c = layout.c
    _size(stats, c.num_pages * c.num_kv_heads * (c.page_size // 16) * 2 * c.head_dim, "stats")
    _size(layout.block_table, B * c.max_pages_per_req, "block_table")
    _size(q, B * Hq * c.head_dim, "q"); _size(seq_lens, B, "seq_lens")
    _size(head_kind, c.num_kv_heads, "head_kind")
    _size(selected, B * c.num_kv_heads * top_k, "selected")
    if selected_phys is not None:
        _size(selected_phys, B * c.num_kv_heads * top_k, "selected_phys")
    here = _layout_device(layout, q)
    _check(load_library().dattn_page_select(
        ctypes.byref(layout.c), _at(stats, here), _at(q, here), B, Hq, _at(seq_lens, here),
        _at(head_kind, here), top_k, _at(selected, here), _at(selected_phys, here),
        _at(ws.buffer, here), ws.buffer.numel(), num_splits, _at(dev_err, here),
        _stream_on(stream, here)), "dattn_page_select")
