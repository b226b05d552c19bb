"""GB300 (sm_103a) sparse-attention decode step: Python binding of libssa_gb300.so.

The calls keep their C names, check what a pointer cannot show (strides, types,
devices, where a wrong one would be misread) and marshal arguments (torch
tensors -> raw pointers, the current CUDA stream); every step of the path runs
in the library's CUDA kernels.  PyTorch provides device
memory, pinned host memory and streams.  There is no CPU fallback: if the
library is missing or no GPU is present the calls raise.

    ssa_store_kv_mirror      write path: quantise/store K,V, mirror, slab
    ssa_index_topk           int8 indexer + top-k page selection
    ssa_ensure_resident      device LRU + miss fetch from the host mirror
    ssa_remap_block_table    logical -> physical block table
    ssa_sparse_paged_decode  attention over the selected pages
    ssa_prefetch_pages       top-k preload of the next step's likely pages
    ssa_rope                 rotary positions of queries and new keys
    ssa_norm_rope            the same with the heads' norms in front
    ssa_prompt_attention     attention over whole prompts, packed sequences
    ssa_beam_select          the next tokens of beams, their states reordered
    ssa_copy_pages, ssa_fork_requests, ssa_compact_pages
                             owners of the pages: copy, fork / grow / free, compact
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssa_gb300.so")

SSA_KV_BF16 = 0
SSA_KV_FP8_E4M3 = 1
SSA_KV_E4M3_PAGE_HEAD = 2
SSA_KV_INT8_PAGE_HEAD = 3
KV_FORMATS = {"bf16": SSA_KV_BF16, "fp8": SSA_KV_FP8_E4M3,
              "e4m3_page_head": SSA_KV_E4M3_PAGE_HEAD, "int8_page_head": SSA_KV_INT8_PAGE_HEAD}

ST_DROP, ST_BAD_ID, ST_MISS_NO_MIRROR, ST_UNRESOLVED, ST_BAD_POS, ST_TIMEOUT = 1, 2, 4, 8, 16, 32
ST_INTERNAL, ST_NO_PAGES = 64, 128

EXPORTS = ("ssa_workspace_size", "ssa_lru_init", "ssa_store_kv_mirror", "ssa_index_topk",
           "ssa_ensure_resident", "ssa_remap_block_table", "ssa_sparse_paged_decode",
           "ssa_status_str", "ssa_last_cuda_error", "ssa_launch_count",
           "ssa_index_topk_static_scratch", "ssa_selftest_bounded_wait", "ssa_host_read_probe",
           "ssa_prefetch_pages", "ssa_ensure_remap", "ssa_sparse_paged_decode_host_tail",
           "ssa_ensure_remap_shared", "ssa_ensure_remap_deferred",
           "ssa_sparse_paged_decode_fetch", "ssa_ensure_remap_bind", "ssa_fetch_misses",
           "ssa_rope", "ssa_rope_frequencies", "ssa_page_refs", "ssa_copy_pages",
           "ssa_fork_requests", "ssa_compact_pages", "ssa_norm_rope", "ssa_prompt_workspace_size",
           "ssa_prompt_attention", "ssa_beam_workspace_size", "ssa_beam_select")


class SsaError(RuntimeError):
    def __init__(self, code: int, msg: str, cuda: int = 0):
        super().__init__(f"{msg} (code {code}" + (f", cudaError {cuda})" if cuda else ")"))
        self.code = code


class SsaLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "page_size", "n_q_heads", "n_kv_heads", "head_dim", "kv_dtype", "n_layers",
        "logical_pages", "pool_slots", "batch", "max_pages", "block_topk", "max_sel")]


class SsaCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "k_pool", "v_pool", "k_scale", "v_scale", "k_mirror", "v_mirror", "k_scale_mirror",
        "v_scale_mirror", "slab", "slab_scale", "slab_sum", "slab_cnt", "slot_of", "page_of",
        "last_use", "clock")]


class SsaRequests(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("ref", ctypes.c_void_p)]


class SsaRopeTensor(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("in_stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3)]


class SsaPromptTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("stride", ctypes.c_int64 * 2)]


class SsaBeams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("scores", "finished", "history", "hist_len")]


_pack_prompt = struct.Struct("@Pi4x2q").pack    # an SsaPromptTensor's bytes
_pack_rope = struct.Struct("@PPi4x6q").pack     # an SsaRopeTensor's bytes


_lib = None


def lib():
    """The loaded C-ABI library (built by build.py); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run sparse_attention_decode_indexer_gb300/build.py")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, P = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER
        L.ssa_workspace_size.restype = ctypes.c_size_t
        L.ssa_workspace_size.argtypes = [P(SsaLayout)]
        L.ssa_lru_init.restype = i32
        L.ssa_lru_init.argtypes = [P(SsaLayout), P(SsaCache), i32, vp]
        L.ssa_store_kv_mirror.restype = i32
        L.ssa_store_kv_mirror.argtypes = [P(SsaLayout), P(SsaCache), i32, i32, vp, vp, vp, i32,
                                          vp, vp]
        L.ssa_index_topk.restype = i32
        L.ssa_index_topk.argtypes = [P(SsaLayout), P(SsaCache), i32, i32] + [vp] * 9
        L.ssa_ensure_resident.restype = i32
        L.ssa_ensure_resident.argtypes = [P(SsaLayout), P(SsaCache), i32, i32] + [vp] * 8
        L.ssa_remap_block_table.restype = i32
        L.ssa_remap_block_table.argtypes = [P(SsaLayout), P(SsaCache), i32, i32] + [vp] * 5
        L.ssa_sparse_paged_decode.restype = i32
        L.ssa_sparse_paged_decode.argtypes = ([P(SsaLayout), P(SsaCache), i32, i32, vp, vp, vp, vp,
                                               ctypes.c_float, vp, vp, vp, vp])
        L.ssa_status_str.restype = ctypes.c_char_p
        L.ssa_status_str.argtypes = [i32]
        L.ssa_last_cuda_error.restype = i32
        L.ssa_last_cuda_error.argtypes = []
        L.ssa_launch_count.restype = ctypes.c_longlong
        L.ssa_launch_count.argtypes = []
        L.ssa_selftest_bounded_wait.restype = i32
        L.ssa_selftest_bounded_wait.argtypes = [vp, vp]
        L.ssa_sparse_paged_decode_host_tail.restype = i32
        L.ssa_sparse_paged_decode_host_tail.argtypes = ([P(SsaLayout), P(SsaCache), i32, i32, vp,
                                                         vp, vp, vp, ctypes.c_float, vp, vp, vp,
                                                         vp])
        L.ssa_ensure_remap_deferred.restype = i32
        L.ssa_ensure_remap_deferred.argtypes = [P(SsaLayout), P(SsaCache), i32, i32] + [vp] * 9
        L.ssa_sparse_paged_decode_fetch.restype = i32
        L.ssa_sparse_paged_decode_fetch.argtypes = ([P(SsaLayout), P(SsaCache), i32, i32, vp, vp,
                                                     vp, vp, vp, ctypes.c_float, vp, vp, vp, vp])
        L.ssa_ensure_remap_bind.restype = i32
        L.ssa_ensure_remap_bind.argtypes = [P(SsaLayout), P(SsaCache), i32, i32] + [vp] * 8
        L.ssa_fetch_misses.restype = i32
        L.ssa_fetch_misses.argtypes = [P(SsaLayout), P(SsaCache), i32, i32] + [vp] * 5
        L.ssa_ensure_remap_shared.restype = i32
        L.ssa_ensure_remap_shared.argtypes = [P(SsaLayout), P(SsaCache), i32, i32] + [vp] * 9
        L.ssa_ensure_remap.restype = i32
        L.ssa_ensure_remap.argtypes = [P(SsaLayout), P(SsaCache), i32, i32] + [vp] * 9
        L.ssa_prefetch_pages.restype = i32
        L.ssa_prefetch_pages.argtypes = ([P(SsaLayout), P(SsaCache), i32, i32, vp, vp, vp, i32]
                                         + [vp] * 6)
        L.ssa_host_read_probe.restype = i32
        L.ssa_host_read_probe.argtypes = [vp, vp, vp, i32, i32, i32, vp]
        f64 = ctypes.c_double
        L.ssa_rope.restype = i32
        L.ssa_rope.argtypes = [i32, i32, i32, i32, i32, vp, ctypes.c_float, i32, i32, vp, i32,
                               ctypes.c_int64, vp, vp, vp]
        L.ssa_norm_rope.restype = i32
        L.ssa_norm_rope.argtypes = [i32, i32, i32, i32, vp, ctypes.c_float, i32, i32, vp, i32,
                                    ctypes.c_int64, vp, vp, vp, vp, ctypes.c_int64,
                                    ctypes.c_float, vp]
        L.ssa_rope_frequencies.restype = i32
        L.ssa_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64,
                                           P(ctypes.c_uint64), P(f64)]
        R = P(SsaRequests)
        L.ssa_page_refs.restype = i32
        L.ssa_page_refs.argtypes = [P(SsaLayout), R, vp, vp]
        L.ssa_copy_pages.restype = i32
        L.ssa_copy_pages.argtypes = [P(SsaLayout), P(SsaCache), vp, vp, i32, vp, vp, vp]
        L.ssa_fork_requests.restype = i32
        L.ssa_fork_requests.argtypes = [P(SsaLayout), P(SsaCache), R, vp, vp, vp, vp, vp]
        L.ssa_compact_pages.restype = i32
        L.ssa_compact_pages.argtypes = [P(SsaLayout), P(SsaCache), R, vp, vp, vp, vp, vp, vp]
        L.ssa_prompt_workspace_size.restype = ctypes.c_size_t
        L.ssa_prompt_workspace_size.argtypes = []
        L.ssa_prompt_attention.restype = i32
        L.ssa_prompt_attention.argtypes = ([i32] * 5 + [vp] * 6 + [i32, ctypes.c_float] + [vp] * 4)
        L.ssa_beam_workspace_size.restype = ctypes.c_size_t
        L.ssa_beam_workspace_size.argtypes = [i32, i32]
        L.ssa_beam_select.restype = i32
        L.ssa_beam_select.argtypes = [i32, i32, i32, i32, vp, ctypes.c_int64, P(SsaBeams),
                                      P(SsaBeams), i32, i32] + [vp] * 7
        _lib = L
    return _lib


def status_str(code: int) -> str:
    return lib().ssa_status_str(int(code)).decode()


def _check(code: int):
    if code != 0:
        raise SsaError(code, status_str(code), lib().ssa_last_cuda_error())


def _ptr(t):
    """A tensor's address (None for a null pointer)."""
    return None if t is None else t.data_ptr()


def _stream(stream):
    """A stream's handle; the current stream's without building a Stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def max_sel_pages(block_topk: int) -> int:
    """Selection width and per-request pool reservation: 2*block_topk + 8."""
    return 2 * block_topk + 8


# ---------------------------------------------------------------------------
# layout and cache (device memory through torch; mirror in pinned host memory)
# ---------------------------------------------------------------------------

@dataclass
class Layout:
    """Shapes of a cache and its calls.  ``kv_format`` names the KV format:
    "bf16", "fp8" (e4m3, one scale per token), "e4m3_page_head" or
    "int8_page_head" (8-bit codes, one K and one V scale per page and KV
    head); None takes bf16 or fp8 by ``fp8``.  Where it is given, ``fp8`` says
    whether the codes are 8 bits wide (V d-major in the pool, with scales),
    and follows it."""
    page_size: int
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    fp8: bool
    n_layers: int
    logical_pages: int
    pool_slots: int
    batch: int
    max_pages: int
    block_topk: int
    kv_format: str | None = None

    def __setattr__(self, name, value):
        # the two never contradict each other: a cache's buffers go by both
        if name == "kv_format" and value is not None:
            if value not in KV_FORMATS:
                raise ValueError(f"kv_format {value!r}: one of {sorted(KV_FORMATS)}")
            object.__setattr__(self, "fp8", value != "bf16")
        elif name == "fp8" and self.kv_format is not None and bool(value) != (self.kv_format != "bf16"):
            raise ValueError(f"fp8 {value!r}: kv_format is {self.kv_format!r}")
        object.__setattr__(self, name, value)

    @property
    def scale_floats(self) -> int:
        """fp32 K scales (and as many V scales) of one page."""
        if self.kv_format in ("e4m3_page_head", "int8_page_head"):
            return self.n_kv_heads
        return self.page_size if self.fp8 else 0

    @property
    def max_sel(self) -> int:
        return max_sel_pages(self.block_topk)

    def c(self) -> SsaLayout:
        return SsaLayout(self.page_size, self.n_q_heads, self.n_kv_heads, self.head_dim,
                         KV_FORMATS[self.kv_format or ("fp8" if self.fp8 else "bf16")],
                         self.n_layers,
                         self.logical_pages, self.pool_slots, self.batch, self.max_pages,
                         self.block_topk, self.max_sel)


def ssa_workspace_size(layout: Layout) -> int:
    lay = layout.c()
    return int(lib().ssa_workspace_size(ctypes.byref(lay)))


class KVCache:
    """Owns the tensors behind one ssa_cache: the paged pool and its scales,
    the optional pinned host mirror, the indexer slab and the LRU state.
    Pool and mirror start zeroed so that rows never written (the tail of a
    request's last page) hold defined bytes; the kernels do not rely on it."""

    def __init__(self, layout: Layout, host_tier: bool, device="cuda"):
        self.layout = layout
        L, Lp, S = layout.n_layers, layout.logical_pages, layout.pool_slots
        H, P, D = layout.n_kv_heads, layout.page_size, layout.head_dim
        esz = 1 if layout.fp8 else 2
        ns = layout.scale_floats
        pb = H * P * D * esz
        u8 = torch.uint8
        self.k_pool = torch.zeros((L, S, pb), dtype=u8, device=device)
        self.v_pool = torch.zeros((L, S, pb), dtype=u8, device=device)
        if layout.fp8:
            self.k_scale = torch.zeros((L, S, ns), dtype=torch.float32, device=device)
            self.v_scale = torch.zeros((L, S, ns), dtype=torch.float32, device=device)
        else:
            self.k_scale = self.v_scale = None
        if host_tier:
            self.k_mirror = torch.zeros((L, Lp, pb), dtype=u8, pin_memory=True)
            self.v_mirror = torch.zeros((L, Lp, pb), dtype=u8, pin_memory=True)
            if layout.fp8:
                self.k_scale_mirror = torch.zeros((L, Lp, ns), dtype=torch.float32, pin_memory=True)
                self.v_scale_mirror = torch.zeros((L, Lp, ns), dtype=torch.float32, pin_memory=True)
            else:
                self.k_scale_mirror = self.v_scale_mirror = None
        else:
            self.k_mirror = self.v_mirror = self.k_scale_mirror = self.v_scale_mirror = None
        self.slab = torch.empty((L, Lp, H * D), dtype=torch.int8, device=device)
        self.slab_scale = torch.empty((L, Lp), dtype=torch.float32, device=device)
        self.slab_sum = torch.empty((L, Lp, H * D), dtype=torch.float32, device=device)
        self.slab_cnt = torch.empty((L, Lp), dtype=torch.int32, device=device)
        self.slot_of = torch.empty((L, Lp), dtype=torch.int32, device=device)
        self.page_of = torch.empty((L, S), dtype=torch.int32, device=device)
        self.last_use = torch.empty((L, S), dtype=torch.int32, device=device)
        self.clock = torch.empty((L,), dtype=torch.int32, device=device)
        self._c = SsaCache(*[ctypes.c_void_p(t.data_ptr()) if t is not None else None for t in (
            self.k_pool, self.v_pool, self.k_scale, self.v_scale, self.k_mirror, self.v_mirror,
            self.k_scale_mirror, self.v_scale_mirror, self.slab, self.slab_scale, self.slab_sum,
            self.slab_cnt, self.slot_of, self.page_of, self.last_use, self.clock)])
        self._lay = layout.c()
        self._row = H * D                # elements of a token's K, and of its V

    @property
    def c(self) -> SsaCache:
        return self._c


# ---------------------------------------------------------------------------
# the calls
# ---------------------------------------------------------------------------

def ssa_lru_init(cache: KVCache, identity: bool, stream=None):
    _check(lib().ssa_lru_init(ctypes.byref(cache._lay), ctypes.byref(cache.c), int(identity),
                              _stream(stream)))


_BF16, _INT64 = torch.bfloat16, torch.int64


def ssa_store_kv_mirror(cache: KVCache, layer0: int, n_layers: int, k, v, pos, status,
                        stream=None):
    """k, v: bf16 [n_layers][T][Hkv][D] (or its bits in an integer type); pos:
    int64 [T] logical token ids; all contiguous."""
    T = pos.shape[0]
    n = n_layers * T * cache._row
    if not (k.is_contiguous() and v.is_contiguous() and pos.is_contiguous() and
            (k.dtype is _BF16 or not k.is_floating_point()) and
            (v.dtype is _BF16 or not v.is_floating_point()) and pos.dtype is _INT64 and
            k.nbytes >= 2 * n and v.nbytes >= 2 * n):
        got = ", ".join(f"{name} {tuple(x.shape)} {x.dtype} strides {x.stride()}"
                        for name, x in (("k", k), ("v", v), ("pos", pos)))
        raise ValueError("k, v: contiguous bfloat16 [n_layers][T][Hkv][D], pos: contiguous int64 "
                         f"[T]; got {got}")
    _check(lib().ssa_store_kv_mirror(cache._lay, cache._c, layer0, n_layers, k.data_ptr(),
                                     v.data_ptr(), pos.data_ptr(), T, _ptr(status),
                                     _stream(stream)))


def ssa_index_topk(cache: KVCache, layer0: int, n_layers: int, q, block_table, seq_lens, sel,
                   n_sel, scores, status, ws, stream=None):
    _check(lib().ssa_index_topk(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                n_layers, _ptr(q), _ptr(block_table), _ptr(seq_lens), _ptr(sel),
                                _ptr(n_sel), _ptr(scores), _ptr(status), _ptr(ws),
                                _stream(stream)))


def ssa_ensure_resident(cache: KVCache, layer0: int, n_layers: int, sel, block_table, miss_page,
                        miss_slot, n_miss, status, ws, stream=None):
    _check(lib().ssa_ensure_resident(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                     n_layers, _ptr(sel), _ptr(block_table), _ptr(miss_page),
                                     _ptr(miss_slot), _ptr(n_miss), _ptr(status), _ptr(ws),
                                     _stream(stream)))


def ssa_ensure_remap(cache: KVCache, layer0: int, n_layers: int, sel, block_table, phys,
                     miss_page, miss_slot, n_miss, status, ws, stream=None):
    """ssa_ensure_resident that also writes the remapped table (one launch fewer)."""
    _check(lib().ssa_ensure_remap(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                  n_layers, _ptr(sel), _ptr(block_table), _ptr(phys),
                                  _ptr(miss_page), _ptr(miss_slot), _ptr(n_miss), _ptr(status),
                                  _ptr(ws), _stream(stream)))


def ssa_ensure_remap_bind(cache: KVCache, layer0: int, n_layers: int, sel, block_table, phys,
                          miss_page, miss_slot, n_miss, status, stream=None):
    """ssa_ensure_remap without the copy: state, phys and the miss lists are
    final; ssa_fetch_misses copies the misses, per layer range, afterwards."""
    _check(lib().ssa_ensure_remap_bind(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                       n_layers, _ptr(sel), _ptr(block_table), _ptr(phys),
                                       _ptr(miss_page), _ptr(miss_slot), _ptr(n_miss),
                                       _ptr(status), _stream(stream)))


def ssa_fetch_misses(cache: KVCache, layer0: int, n_layers: int, miss_page, miss_slot, n_miss,
                     status, stream=None):
    """Copy the listed misses of layers [layer0, layer0 + n_layers) mirror ->
    slot; the lists are those ssa_ensure_remap_bind wrote for these layers."""
    _check(lib().ssa_fetch_misses(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                  n_layers, _ptr(miss_page), _ptr(miss_slot), _ptr(n_miss),
                                  _ptr(status), _stream(stream)))


def ssa_ensure_remap_deferred(cache: KVCache, layer0: int, n_layers: int, sel, block_table, phys,
                              miss_page, miss_slot, n_miss, status, ws, stream=None):
    """The ensure's state update and remap without the copy: misses marked
    -2 - slot in phys, for ssa_sparse_paged_decode_fetch to fetch."""
    _check(lib().ssa_ensure_remap_deferred(ctypes.byref(cache._lay), ctypes.byref(cache.c),
                                           layer0, n_layers, _ptr(sel), _ptr(block_table),
                                           _ptr(phys), _ptr(miss_page), _ptr(miss_slot),
                                           _ptr(n_miss), _ptr(status), _ptr(ws), _stream(stream)))


def ssa_sparse_paged_decode_fetch(cache: KVCache, layer0: int, n_layers: int, q, sel, phys,
                                  block_table, seq_lens, sm_scale: float, out, status, ws,
                                  stream=None):
    """Attention that fetches the pages ssa_ensure_remap_deferred marked from
    the host mirror and writes them into their slots as it goes."""
    _check(lib().ssa_sparse_paged_decode_fetch(
        ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0, n_layers, _ptr(q), _ptr(sel),
        _ptr(phys), _ptr(block_table), _ptr(seq_lens), float(sm_scale), _ptr(out), _ptr(status),
        _ptr(ws), _stream(stream)))


def ssa_ensure_remap_shared(cache: KVCache, layer0: int, n_layers: int, sel, block_table, phys,
                            miss_page, miss_slot, n_miss, status, ws, stream=None):
    """One residency for the layer range (layer0's state): the union of the
    layers' selections ensured, each miss copied for every layer, phys for
    every layer."""
    _check(lib().ssa_ensure_remap_shared(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                         n_layers, _ptr(sel), _ptr(block_table), _ptr(phys),
                                         _ptr(miss_page), _ptr(miss_slot), _ptr(n_miss),
                                         _ptr(status), _ptr(ws), _stream(stream)))


def ssa_prefetch_pages(cache: KVCache, layer0: int, n_layers: int, scores, block_table,
                       seq_lens, width: int, fetch_page, fetch_slot, n_fetch, status, ws,
                       stream=None):
    """Top-k preload after a step's ensure: fetch the top (width-1) pages plus
    the last page of each request by that step's scores ahead of the next."""
    _check(lib().ssa_prefetch_pages(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                    n_layers, _ptr(scores), _ptr(block_table), _ptr(seq_lens),
                                    int(width), _ptr(fetch_page), _ptr(fetch_slot),
                                    _ptr(n_fetch), _ptr(status), _ptr(ws), _stream(stream)))


def ssa_remap_block_table(cache: KVCache, layer0: int, n_layers: int, sel, block_table, phys,
                          status, stream=None):
    _check(lib().ssa_remap_block_table(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                       n_layers, _ptr(sel), _ptr(block_table), _ptr(phys),
                                       _ptr(status), _stream(stream)))


def ssa_sparse_paged_decode(cache: KVCache, layer0: int, n_layers: int, q, sel, phys, seq_lens,
                            sm_scale: float, out, status, ws, stream=None):
    _check(lib().ssa_sparse_paged_decode(ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0,
                                         n_layers, _ptr(q), _ptr(sel), _ptr(phys),
                                         _ptr(seq_lens), float(sm_scale), _ptr(out),
                                         _ptr(status), _ptr(ws), _stream(stream)))


def ssa_sparse_paged_decode_host_tail(cache: KVCache, layer0: int, n_layers: int, q, sel,
                                      block_table, seq_lens, sm_scale: float, out, status, ws,
                                      stream=None):
    """Attention over the selected pages, non-resident ones read straight from
    the pinned host mirror (no ensure, no copy)."""
    _check(lib().ssa_sparse_paged_decode_host_tail(
        ctypes.byref(cache._lay), ctypes.byref(cache.c), layer0, n_layers, _ptr(q), _ptr(sel),
        _ptr(block_table), _ptr(seq_lens), float(sm_scale), _ptr(out), _ptr(status), _ptr(ws),
        _stream(stream)))


# ---------------------------------------------------------------------------
# owners of the pages
# ---------------------------------------------------------------------------

def _on_current_device(device: int):
    """The calls launch on the current device: refuse tensors of another (by
    ordinal, -1 for the host)."""
    if device < 0 or device != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on device {device}, which is not the current CUDA device")


def _ints(name, t, n, device: int):
    """The address of a contiguous int32 tensor of n entries on a device
    (ordinal), or an error."""
    if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous() or \
            t.get_device() != device:
        raise ValueError(f"{name}: {n} contiguous int32 on device {device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


class RequestTable:
    """The requests' pages: block_table [B][max_pages], seq_lens [B] and the
    references of every logical page, ref [logical_pages], all int32 on the
    device.  Contiguous int32 tensors already there are taken as they are, so
    that a runner's tables change in place.  Without ``ref`` the rows are counted
    (ssa_page_refs); add to ref[p] to pin page p."""

    def __init__(self, layout: Layout, block_table, seq_lens, ref=None, device="cuda"):
        i32 = torch.int32
        self.layout = layout
        self.block_table = torch.as_tensor(block_table).to(device=device, dtype=i32).contiguous()
        self.seq_lens = torch.as_tensor(seq_lens).to(device=device, dtype=i32).contiguous()
        dev = self.block_table.get_device()
        _ints("block_table", self.block_table, layout.batch * layout.max_pages, dev)
        _ints("seq_lens", self.seq_lens, layout.batch, dev)
        if ref is None:
            self.ref = torch.zeros((layout.logical_pages,), dtype=i32, device=device)
        else:
            self.ref = torch.as_tensor(ref).to(device=device, dtype=i32).contiguous()
        _ints("ref", self.ref, layout.logical_pages, dev)
        self._c = SsaRequests(self.block_table.data_ptr(), self.seq_lens.data_ptr(),
                              self.ref.data_ptr())
        self._lay = layout.c()
        if ref is None:
            ssa_page_refs(self)


def _same_pages(cache: KVCache, table: RequestTable):
    a, b = cache.layout, table.layout
    if (a.batch, a.max_pages, a.logical_pages, a.page_size) != \
            (b.batch, b.max_pages, b.logical_pages, b.page_size):
        raise ValueError("the cache and the request table have different layouts")
    if cache.slot_of.get_device() != table.ref.get_device():
        raise ValueError("the cache and the request table are on different devices")


def ssa_page_refs(table: RequestTable, status=None, stream=None):
    """Count the rows' references anew (any pins are forgotten)."""
    _on_current_device(table.ref.get_device())
    _check(lib().ssa_page_refs(table._lay, table._c, _ptr(status), _stream(stream)))


def ssa_copy_pages(cache: KVCache, src, dst, status, ws, stream=None):
    """Page dst[i] := page src[i] in every layer; int32 device lists, negative
    ids are padding."""
    n, dev = src.numel(), cache.slot_of.get_device()
    src, dst = _ints("src", src, n, dev), _ints("dst", dst, n, dev)
    _on_current_device(dev)
    _check(lib().ssa_copy_pages(cache._lay, cache._c, src, dst, n, _ptr(status), _ptr(ws),
                                _stream(stream)))


def ssa_fork_requests(cache: KVCache, table: RequestTable, parent, new_lens, status, ws,
                      stream=None):
    """Row i continues what row parent[i] held (-1: nothing, the row is freed),
    grown to new_lens[i] tokens (None: no growth): full pages shared, partly
    filled ones copied, new ones taken, unused ones freed."""
    _same_pages(cache, table)
    B, dev = cache.layout.batch, cache.slot_of.get_device()
    parent = _ints("parent", parent, B, dev)
    new_lens = None if new_lens is None else _ints("new_lens", new_lens, B, dev)
    _on_current_device(dev)
    _check(lib().ssa_fork_requests(cache._lay, cache._c, table._c, parent, new_lens, _ptr(status),
                                   _ptr(ws), _stream(stream)))


def ssa_compact_pages(cache: KVCache, table: RequestTable, status, ws, moved_from=None,
                      moved_to=None, n_moved=None, stream=None):
    """Move the live pages to the lowest ids; the moves go to moved_from /
    moved_to ([logical_pages]) and their number to n_moved ([1])."""
    _same_pages(cache, table)
    Lp, dev = cache.layout.logical_pages, cache.slot_of.get_device()
    outs = [None if t is None else _ints(name, t, n, dev) for name, t, n in (
        ("moved_from", moved_from, Lp), ("moved_to", moved_to, Lp), ("n_moved", n_moved, 1))]
    _on_current_device(dev)
    _check(lib().ssa_compact_pages(cache._lay, cache._c, table._c, *outs, _ptr(status), _ptr(ws),
                                   _stream(stream)))


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}
_ROPE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


@dataclass
class RopeScaling:
    """How the frequencies change for contexts longer than ``original_len``:
    "linear" and "ntk" take ``factor``; "bands" and "yarn" also
    ``original_len`` and the turns over it, ``low`` and ``high``, between
    which pairs go from stretched to kept (include/ssa.h has the formulas)."""
    kind: str
    factor: float = 1.0
    original_len: float = 0.0
    low: float = 1.0
    high: float = 32.0


class RopePlan:
    """Frequencies of ssa_rope on the device.

    head_dim, rotary_dim (default: the whole head), interleaved: the layout of
    a head's pairs.  base and scaling give the frequencies, or ``theta``
    (radians per position of each pair) gives them outright.  factor: the
    factor on cos and sin (default: the scaling's)."""

    def __init__(self, head_dim: int, rotary_dim: int | None = None, base: float = 10000.0,
                 interleaved: bool = False, scaling: RopeScaling | None = None, theta=None,
                 factor: float | None = None, device="cuda"):
        rd = head_dim if rotary_dim is None else rotary_dim
        if rd < 2 or rd % 2 or rd > head_dim:
            raise ValueError(f"rotary_dim {rd}: an even number from 2 to head_dim {head_dim}")
        self.head_dim, self.rotary_dim, self.interleaved = head_dim, rd, bool(interleaved)
        own = ctypes.c_double(1.0)
        if theta is not None:
            theta = [float(x) for x in theta]
            if len(theta) != rd // 2 or not all(math.isfinite(x) for x in theta):
                raise ValueError(f"theta: {rd // 2} finite numbers")
            freq = [round(math.ldexp(math.fmod(x / (2 * math.pi), 1.0), 64)) % (1 << 64)
                    for x in theta]
        else:
            sc = scaling or RopeScaling("plain")
            if sc.kind not in ROPE_SCALINGS:
                raise ValueError(f"scaling {sc.kind!r}: one of {sorted(ROPE_SCALINGS)}")
            buf = (ctypes.c_uint64 * (rd // 2))()
            _check(lib().ssa_rope_frequencies(rd, float(base), ROPE_SCALINGS[sc.kind],
                                              float(sc.factor), float(sc.original_len),
                                              float(sc.low), float(sc.high), buf,
                                              ctypes.byref(own)))
            freq = list(buf)
        self.factor = float(own.value if factor is None else factor)
        # two's complement: the same 64 bits
        self.freq = torch.tensor([f - (1 << 64) if f >= 1 << 63 else f for f in freq],
                                 dtype=torch.int64, device=device)
        self._freq, self._dev = self.freq.data_ptr(), self.freq.get_device()


def _rope_tensor(plan, name, x, out, shape):
    """The C view of one tensor, whose shape but for the heads is `shape`:
    any strides but the last."""
    if out is None:
        out = x
    got, lead = x.shape, len(shape) == 4
    # (entry by entry: slices of sizes cost more than the rest of a small call)
    if len(got) != len(shape) or got[0] != shape[0] or got[-1] != shape[-1] or \
            (lead and got[1] != shape[1]):
        raise ValueError(f"{name}: [n_layers][T][heads][D] or [T][heads][D] with (T, D) of the "
                         f"positions and the plan and the same layers for q and k, got "
                         f"{tuple(got)}")
    st = x.stride()
    so = st if out is x else out.stride()
    if out is not x and (out.shape != got or out.dtype != x.dtype or
                         out.get_device() != plan._dev):
        raise ValueError(f"{name}_out: shape, type or device other than {name}'s")
    if st[-1] != 1 or so[-1] != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return _pack_rope(x.data_ptr(), out.data_ptr(), got[-2], st[0] if lead else 0, st[-3], st[-2],
                      so[0] if lead else 0, so[-3], so[-2])


def _rope_args(plan, positions, q, k, q_out, k_out):
    """Checked arguments of a call on q and k: type, layers, tokens, 64-bit
    positions or not, the C views."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k")
    dtype = _ROPE_DTYPES.get(x.dtype)
    if dtype is None or (k is not None and k.dtype != x.dtype):
        raise ValueError("q and k: bfloat16, float16 or float32, the same")
    wide = positions.dtype == torch.int64
    if positions.dim() != 1 or not (wide or positions.dtype == torch.int32) or \
            not positions.is_contiguous():
        raise ValueError("positions: a contiguous [T] int32 or int64 tensor")
    dev = plan._dev
    if x.get_device() != dev or positions.get_device() != dev or \
            (k is not None and k.get_device() != dev):
        raise ValueError(f"q, k and positions: on the plan's device, {plan.freq.device}")
    T = positions.shape[0]
    shape = (x.shape[0], T, 0, plan.head_dim) if x.dim() == 4 else (T, 0, plan.head_dim)
    cq = _rope_tensor(plan, "q", q, q_out, shape) if q is not None else None
    ck = _rope_tensor(plan, "k", k, k_out, shape) if k is not None else None
    return dtype, shape[0] if len(shape) == 4 else 1, T, wide, cq, ck


def ssa_rope(plan: RopePlan, positions, q=None, k=None, q_out=None, k_out=None, offset: int = 0,
             inverse: bool = False, stream=None):
    """Rotate q and k ([n_layers][T][heads][D] or [T][heads][D], strided views
    allowed) by positions + offset ([T] int32 or int64), in place or into
    q_out / k_out; one launch for both.  ``inverse`` turns back (the gradient
    of the rotation)."""
    dtype, n_layers, T, wide, cq, ck = _rope_args(plan, positions, q, k, q_out, k_out)
    if T == 0 or n_layers == 0:
        return
    _on_current_device(plan._dev)
    _check(lib().ssa_rope(dtype, plan.head_dim, plan.rotary_dim, plan.interleaved, inverse,
                          plan._freq, plan.factor, n_layers, T, positions.data_ptr(), wide,
                          offset, cq, ck, _stream(stream)))


class HeadNorm:
    """Norm of every head of q and k: x / sqrt(mean(x^2) + eps) * (weight + offset).

    q_weight, k_weight: [D], or [n_layers][D] for a vector per layer, kept as
    fp32 on the device; None: ones.  ``offset``: 1 for models whose weights are
    kept about zero."""

    def __init__(self, q_weight=None, k_weight=None, eps: float = 1e-6, offset: float = 0.0,
                 device="cuda"):
        ws = [None if w is None else
              (torch.as_tensor(w).detach().to(device=device, dtype=torch.float32) + offset).contiguous()
              for w in (q_weight, k_weight)]
        shapes = {tuple(w.shape) for w in ws if w is not None}
        if len(shapes) > 1 or any(len(x) not in (1, 2) for x in shapes):
            raise ValueError("q_weight, k_weight: [D] or [n_layers][D], the same for both")
        if not 0.0 <= eps < math.inf:
            raise ValueError(f"eps {eps!r}: a finite number, not negative")
        if offset and None in ws and shapes:
            raise ValueError("offset: of both weights, so both of them or none")
        self.q_weight, self.k_weight = ws
        self.eps = float(eps)
        shape = shapes.pop() if shapes else None
        self.layers = shape[0] if shape and len(shape) == 2 else None     # None: shared by all
        self.head_dim = shape[-1] if shape else None
        self._ptr = [0 if w is None else w.data_ptr() for w in ws]
        self._dev = next((w.get_device() for w in ws if w is not None), None)

    def __setattr__(self, name, value):
        # calls go by the addresses of the weights made above
        if name in ("q_weight", "k_weight") and "_ptr" in self.__dict__:
            raise AttributeError(f"{name}: change the tensor in place (copy_, fill_)")
        object.__setattr__(self, name, value)


def ssa_norm_rope(plan: RopePlan, norm: HeadNorm, positions, q=None, k=None, q_out=None,
                  k_out=None, offset: int = 0, layer0: int = 0, stream=None):
    """ssa_rope with the heads' norms in front of the rotation, in the same
    pass.  layer0: the layer of the first slice of q and k, where the norm has a
    weight vector per layer."""
    dtype, n_layers, T, wide, cq, ck = _rope_args(plan, positions, q, k, q_out, k_out)
    D = plan.head_dim
    if norm.head_dim not in (None, D) or norm._dev not in (None, plan._dev):
        raise ValueError(f"norm: weights of {norm.head_dim} on device {norm._dev}, the plan's heads "
                         f"are {D} on {plan._dev}")
    step = 0
    if norm.layers is not None:
        if layer0 < 0 or layer0 + n_layers > norm.layers:
            raise ValueError(f"layers {layer0} to {layer0 + n_layers} of a norm of {norm.layers}")
        step = D
    if T == 0 or n_layers == 0:
        return
    _on_current_device(plan._dev)
    wq, wk = (w and w + 4 * step * layer0 for w in norm._ptr)
    _check(lib().ssa_norm_rope(dtype, D, plan.rotary_dim, plan.interleaved, plan._freq,
                               plan.factor, n_layers, T, positions.data_ptr(), wide, offset, cq,
                               ck, wq, wk, step, norm.eps, _stream(stream)))


# ---------------------------------------------------------------------------
# attention over whole prompts
# ---------------------------------------------------------------------------

_PROMPT_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def ssa_prompt_workspace_size() -> int:
    """Bytes of scratch of ssa_prompt_attention, whatever the call's sizes."""
    return int(lib().ssa_prompt_workspace_size())


def _refuse_prompt(q, k, v, out):
    """Why ssa_prompt_attention does not take these tensors."""
    for name, x in (("q", q), ("k", k), ("v", v), ("out", out)):
        if x.dim() != 3 or x.dtype != q.dtype or x.get_device() != q.get_device():
            raise ValueError(f"{name}: [tokens][heads][D] of q's type and device, got "
                             f"{tuple(x.shape)} {x.dtype} on {x.device}")
        if x.numel() and x.stride(2) != 1:
            raise ValueError(f"{name}: the elements of a head must be contiguous")
    raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}, out "
                     f"{tuple(out.shape)}: one head size, k and v alike, q and out alike")


def ssa_prompt_attention(q, k, v, cu_q, out, status, ws, cu_k=None, causal: bool = True,
                         sm_scale: float | None = None, lse=None, stream=None):
    """Attention over packed sequences of different lengths: q [Tq][Hq][D] over
    k, v [Tk][Hkv][D] into out [Tq][Hq][D], strided views allowed.  Sequence s
    has the query tokens cu_q[s] .. cu_q[s + 1] and the keys cu_k[s] ..
    cu_k[s + 1] (default: cu_q), int32 on the device; with ``causal`` its query
    tokens are the last ones of its keys.  sm_scale: default 1 / sqrt(D).  lse:
    fp32 [Tq][Hq], the logarithm of each row's sum.  status: one int32, or None.
    ws: at least ssa_prompt_workspace_size() contiguous bytes."""
    # (a small call's time is this function's: each property is read once)
    dt, dev, size, sk = q.dtype, q.get_device(), q.shape, k.shape
    dtype = _PROMPT_DTYPES.get(dt)
    if dtype is None:
        raise ValueError(f"q, k, v: bfloat16 or float16, got {dt}")
    if len(size) != 3 or len(sk) != 3 or size[2] != sk[2] or v.shape != sk or out.shape != size or \
            k.dtype is not dt or v.dtype is not dt or out.dtype is not dt or \
            k.get_device() != dev or v.get_device() != dev or out.get_device() != dev:
        _refuse_prompt(q, k, v, out)
    n_q, heads, D = size
    n_k, heads_k, _ = sk
    q0, q1, q2 = q.stride()
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    o0, o1, o2 = out.stride()
    if (q2 != 1 or o2 != 1) and n_q or (k2 != 1 or v2 != 1) and n_k:
        _refuse_prompt(q, k, v, out)
    n = cu_q.shape[0] if cu_q.dim() == 1 else 0
    pq = _ints("cu_q", cu_q, n, dev)
    pk = pq if cu_k is None or cu_k is cu_q else _ints("cu_k", cu_k, n, dev)
    if n < 1:
        raise ValueError("cu_q: the first token of each sequence, and the end of the last")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != size[:2] or
                            not lse.is_contiguous() or lse.get_device() != dev):
        raise ValueError(f"lse: contiguous float32 [{n_q}][{heads}] on q's device")
    ps = None if status is None else _ints("status", status, 1, dev)
    L = lib()
    if ws.get_device() != dev or not ws.is_contiguous() or \
            ws.nbytes < L.ssa_prompt_workspace_size():
        raise ValueError("ws: ssa_prompt_workspace_size() contiguous bytes on q's device")
    _on_current_device(dev)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    _check(L.ssa_prompt_attention(
        dtype, D, n - 1, n_q, n_k, _pack_prompt(q.data_ptr(), heads, q0, q1),
        _pack_prompt(k.data_ptr(), heads_k, k0, k1), _pack_prompt(v.data_ptr(), heads_k, v0, v1),
        _pack_prompt(out.data_ptr(), heads, o0, o1), pq, pk, causal, sm_scale, _ptr(lse),
        ps, ws.data_ptr(), _stream(stream)))


# ---------------------------------------------------------------------------
# the next tokens
# ---------------------------------------------------------------------------

class BeamState:
    """What beams carry from token to token, ``groups`` times ``beams`` rows:
    scores [B] fp32 (sums of log-probabilities), with ``finished`` a byte per row
    that says it has ended, with ``max_len`` the tokens so far, history
    [B][max_len] and hist_len [groups], int32.  Starts before the first token:
    the first row of a group at 0, the others at -infinity, nothing in the
    histories."""

    def __init__(self, groups: int, beams: int, max_len: int = 0, finished: bool = False,
                 device="cuda"):
        B, i32 = groups * beams, torch.int32
        self.groups, self.beams, self.max_len = groups, beams, max_len
        self.scores = torch.full((groups, beams), -math.inf, device=device)
        self.scores[:, 0] = 0.0
        self.scores = self.scores.view(B)
        self.finished = torch.zeros((B,), dtype=torch.uint8, device=device) if finished else None
        self.history = torch.zeros((B, max_len), dtype=i32, device=device) if max_len else None
        self.hist_len = torch.zeros((groups,), dtype=i32, device=device) if max_len else None
        self._dev = self.scores.get_device()
        self._c = SsaBeams(*[_ptr(t) for t in (self.scores, self.finished, self.history,
                                               self.hist_len)])

    def __setattr__(self, name, value):
        # calls go by the addresses of the tensors made above
        if "_c" in self.__dict__:
            raise AttributeError(f"{name}: change the tensors in place (copy_, fill_)")
        object.__setattr__(self, name, value)


def ssa_beam_workspace_size(groups: int, beams: int) -> int:
    """Bytes of scratch of ssa_beam_select (zeroed once), for any vocabulary and
    for fewer groups or beams too."""
    return int(lib().ssa_beam_workspace_size(groups, beams))


def ssa_beam_select(logits, state: BeamState, parent, token, status, ws, out: BeamState | None = None,
                    eos: int = -1, seq_lens=None, new_lens=None, stream=None):
    """The best (row, token) pairs of every group of beams by score plus
    log-probability: logits [B][V] (rows may be strided), ``state`` before and
    ``out`` after (default: in place); parent and token [B] int32 out, new_lens
    [B] = seq_lens[parent] + 1, as ssa_fork_requests takes parent and new_lens.
    eos: the token that ends a beam (a state with ``finished``), or -1."""
    out = state if out is None else out
    B, dev = state.groups * state.beams, state._dev
    dtype = _ROPE_DTYPES.get(logits.dtype)
    if dtype is None or logits.dim() != 2 or logits.shape[0] != B or logits.get_device() != dev or \
            (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError(f"logits: [{B}][V] bfloat16, float16 or float32 on the state's device, a "
                         f"row's elements contiguous, got {tuple(logits.shape)} {logits.dtype} on "
                         f"{logits.device}")
    if (out.groups, out.beams, out.max_len, out._dev) != \
            (state.groups, state.beams, state.max_len, dev):
        raise ValueError("state and out: of other sizes, or on other devices")
    if (eos >= 0) != (state.finished is not None) or (eos >= 0) != (out.finished is not None):
        raise ValueError(f"eos {eos}: a token for states with finished, -1 for states without")
    if (seq_lens is None) != (new_lens is None):
        raise ValueError("seq_lens and new_lens: both or none")
    ints = [None if t is None else _ints(name, t, n, dev) for name, t, n in (
        ("parent", parent, B), ("token", token, B), ("seq_lens", seq_lens, B),
        ("new_lens", new_lens, B), ("status", status, 1))]
    if ws.get_device() != dev or not ws.is_contiguous() or \
            ws.nbytes < lib().ssa_beam_workspace_size(state.groups, state.beams):
        raise ValueError("ws: ssa_beam_workspace_size(groups, beams) contiguous bytes on the "
                         "state's device")
    _on_current_device(dev)
    _check(lib().ssa_beam_select(dtype, state.groups, state.beams, logits.shape[1],
                                 logits.data_ptr(), logits.stride(0), state._c, out._c,
                                 state.max_len, eos, *ints, ws.data_ptr(), _stream(stream)))


def ssa_selftest_bounded_wait(status, stream=None):
    """One CTA waits on an mbarrier nothing arrives on; the bounded wait gives
    up after about a second and sets ST_TIMEOUT in ``status``."""
    _check(lib().ssa_selftest_bounded_wait(_ptr(status), _stream(stream)))


def ssa_host_read_probe(src, dst, offsets, chunk_bytes: int, loads_per_thread: int = 8,
                        stream=None):
    """Copy chunks of ``src`` (pinned host or device) at the int64 byte
    ``offsets`` (a device tensor) into ``dst`` with SM loads: the host link's
    rate for the access pattern of the miss fetch."""
    _check(lib().ssa_host_read_probe(_ptr(src), _ptr(dst), _ptr(offsets), int(offsets.numel()),
                                     int(chunk_bytes), int(loads_per_thread), _stream(stream)))


def launch_count() -> int:
    return int(lib().ssa_launch_count())
