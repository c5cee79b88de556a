"""Thin ctypes binding of libnexus.so (include/nexus.h). Argument marshalling only:
every step of the eviction path runs in the library's CUDA kernels.

Tensors are torch CUDA tensors; the stream is torch's current stream unless given.
The library must be built (``__graft_entry__.build()`` or
``python -m streaming_kv_cache_step_gb300.build``); if it is missing, every call
raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from dataclasses import dataclass
from fractions import Fraction

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnexus.so")

NX_OK, NX_ERR_INVALID_ARG, NX_ERR_UNSUPPORTED, NX_ERR_CUDA = 0, 1, 2, 3
NX_ERR_TIMEOUT, NX_ERR_WORKSPACE, NX_ERR_DEVICE_FAULT = 4, 5, 6
NX_DEV_TIMEOUT, NX_DEV_BAD_LEN, NX_DEV_BAD_BUDGET, NX_DEV_BAD_PAGE = 1, 2, 4, 8
NX_DEV_BAD_TOKENS, NX_DEV_FULL, NX_DEV_BAD_IMAGE = 16, 32, 64
DTYPE_F32, DTYPE_BF16 = 0, 1
MODE_RESERVOIR, MODE_TOPK = 0, 1

SYMBOLS = ("nexus_workspace_bytes", "nexus_direct_scores", "nexus_walk",
           "nexus_reservoir_select", "kv_compact", "nexus_evict_step", "nx_status_string",
           "nexus_last_launch_count", "nexus_debug_compact", "nexus_last_launch_name",
           "nexus_profile_next_call", "nexus_debug_force_simt", "nexus_debug_set_trace",
           "nexus_debug_scorer_config", "nexus_debug_scorer_layout", "kv_compact_noalloc",
           "nexus_last_scorer", "nexus_debug_compact_kernel", "nexus_append",
           "nexus_append_image", "nexus_quantize", "nexus_attend_workspace_bytes", "nexus_attend")
SCORER_NONE, SCORER_TENSOR_CORE, SCORER_CUDA_CORE, SCORER_TENSOR_CORE_TWO_PASS = 0, 1, 2, 3


class NexusError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class CCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("layers", "seqs", "kv_heads", "group", "head_dim", "capacity", "page_size",
                 "num_pages", "max_pages_per_seq", "dtype")] + [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pos", ctypes.c_void_p),
        ("lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p)]


class CParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("window", "walk_len", "n_sink", "n_recent", "n_avg", "mode")] + [
        ("lam", ctypes.c_float), ("eps_tie", ctypes.c_float), ("budget", ctypes.c_void_p),
        ("budget_max", ctypes.c_int32), ("seq_id_base", ctypes.c_int32),
        ("layer_id_base", ctypes.c_int32), ("step", ctypes.c_uint32), ("seed", ctypes.c_uint64),
        ("block_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("slice_budget", ctypes.c_void_p)]


class CTokens(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("layer", "tokens", "max_tokens", "reserved")] + [
        ("cu_tokens", ctypes.c_void_p)]


class CAppend(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_out", ctypes.c_void_p),
                ("pos", ctypes.c_void_p), ("lens_in", ctypes.c_void_p),
                ("rotary", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("q_norm", ctypes.c_void_p),
                ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class CImage(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "rows")]


class CAttend(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH):
    """Load libnexus.so once; raise if it is not built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libnexus.so is not built ({path}); run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            P = ctypes.c_void_p
            lib.nexus_workspace_bytes.argtypes = [P, P]
            lib.nexus_workspace_bytes.restype = ctypes.c_size_t
            lib.nexus_direct_scores.argtypes = [P, P, P, P, P, P, ctypes.c_size_t, P, P]
            lib.nexus_walk.argtypes = [P, P, P, P, P, P, ctypes.c_size_t, P, P]
            lib.nexus_reservoir_select.argtypes = [P, P, P, P, P, ctypes.c_size_t, P, P]
            lib.kv_compact.argtypes = [P, P, P, P, ctypes.c_size_t, P, P]
            lib.nexus_evict_step.argtypes = [P, P, P, P, P, ctypes.c_size_t, P, P]
            for name in ("nexus_direct_scores", "nexus_walk", "nexus_reservoir_select",
                         "kv_compact", "nexus_evict_step"):
                getattr(lib, name).restype = ctypes.c_int
            lib.nexus_debug_compact.argtypes = [P, P, P, P, ctypes.c_size_t, P, P,
                                                ctypes.c_longlong]
            lib.nexus_debug_compact.restype = ctypes.c_int
            lib.nx_status_string.argtypes = [ctypes.c_int]
            lib.nx_status_string.restype = ctypes.c_char_p
            lib.nexus_last_scorer.argtypes = []
            lib.nexus_last_scorer.restype = ctypes.c_int32
            lib.nexus_last_launch_count.argtypes = []
            lib.nexus_last_launch_count.restype = ctypes.c_int32
            lib.nexus_last_launch_name.argtypes = [ctypes.c_int32]
            lib.nexus_last_launch_name.restype = ctypes.c_char_p
            lib.nexus_profile_next_call.argtypes = [ctypes.c_void_p, ctypes.c_int32]
            lib.nexus_profile_next_call.restype = None
            lib.nexus_debug_force_simt.argtypes = [ctypes.c_int32]
            lib.nexus_debug_force_simt.restype = None
            lib.nexus_debug_compact_kernel.argtypes = [ctypes.c_int32]
            lib.nexus_debug_compact_kernel.restype = None
            lib.nexus_debug_scorer_layout.argtypes = [ctypes.c_int32]
            lib.nexus_debug_scorer_layout.restype = None
            lib.nexus_debug_set_trace.argtypes = [ctypes.c_void_p]
            lib.nexus_debug_set_trace.restype = None
            lib.nexus_debug_scorer_config.argtypes = [ctypes.c_void_p]
            lib.nexus_debug_scorer_config.restype = None
            lib.nexus_append.argtypes = [P, P, P, P, P]
            lib.nexus_append_image.argtypes = [P, P, P, P, P, P]
            lib.nexus_quantize.argtypes = [P, P, P, P, P]
            lib.nexus_attend.argtypes = [P, P, P, P, P, ctypes.c_size_t, P, P]
            for name in ("nexus_append", "nexus_append_image", "nexus_quantize",
                         "nexus_attend"):
                getattr(lib, name).restype = ctypes.c_int
            lib.nexus_attend_workspace_bytes.argtypes = [P, P]
            lib.nexus_attend_workspace_bytes.restype = ctypes.c_size_t
            _lib = lib
    return _lib


def force_simt(on: bool) -> None:
    """Route scoring to the CUDA-core scorer even where the tensor-core one applies."""
    load().nexus_debug_force_simt(1 if on else 0)


COMPACT_AUTO, COMPACT_TILES, COMPACT_SLICES = 0, 1, 2


def compact_kernel(which: int) -> None:
    """Testing hook: the compaction kernel, process-wide (COMPACT_TILES, COMPACT_SLICES or
    COMPACT_AUTO)."""
    load().nexus_debug_compact_kernel(int(which))


def scorer_layout(teams: int) -> None:
    """Tensor-core scorer layout: 2 or 1 pipelines per CTA, 0 for the automatic choice."""
    load().nexus_debug_scorer_layout(int(teams))


def scorer_config() -> dict:
    """Configuration of the last tensor-core scorer launch made from this thread."""
    out = (ctypes.c_int32 * 8)()
    load().nexus_debug_scorer_config(out)
    keys = ("teams_per_cta", "occupancy_api", "grid", "tiles_per_chunk", "tmem_buffers",
            "chunks_per_slice", "tmem_cols", "smem_bytes")
    return dict(zip(keys, list(out)))


def set_trace(buf) -> None:
    """Install (int64 CUDA tensor) or remove (None) the scorer's phase-trace buffer."""
    load().nexus_debug_set_trace(None if buf is None else ctypes.c_void_p(buf.data_ptr()))


def status_string(status: int) -> str:
    return load().nx_status_string(int(status)).decode()


def last_scorer() -> int:
    """SCORER_TENSOR_CORE, SCORER_CUDA_CORE or SCORER_NONE for the last call of this thread."""
    return int(load().nexus_last_scorer())


def last_launch_count() -> int:
    return int(load().nexus_last_launch_count())


def last_launch_names() -> list[str]:
    lib = load()
    return [lib.nexus_last_launch_name(i).decode() for i in range(last_launch_count())]


def profile_next_call(events) -> object:
    """Arm per-launch events (torch.cuda.Event with timing) for the next call; returns
    the ctypes array, which the caller keeps alive until that call returns."""
    for e in events:
        if not e.cuda_event:          # torch creates the CUDA event on first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    load().nexus_profile_next_call(arr, len(events))
    return arr


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without a Stream object around it (2.7 us less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


@dataclass
class Cache:
    """Device KV cache in the layouts of include/nexus.h (tensors stay owned by torch)."""
    k: torch.Tensor
    v: torch.Tensor
    pos: torch.Tensor
    lens: torch.Tensor
    layers: int
    seqs: int
    kv_heads: int
    group: int
    head_dim: int
    capacity: int
    page_size: int = 0
    num_pages: int = 0
    max_pages_per_seq: int = 0
    block_table: torch.Tensor | None = None

    @classmethod
    def from_dict(cls, d: dict) -> "Cache":
        return cls(k=d["k"], v=d["v"], pos=d["pos"], lens=d["lens"], layers=d["layers"],
                   seqs=d["seqs"], kv_heads=d["kv_heads"], group=d["group"],
                   head_dim=d["head_dim"], capacity=d["capacity"],
                   page_size=d.get("page_size", 0), num_pages=d.get("num_pages", 0),
                   max_pages_per_seq=d.get("max_pages_per_seq", 0),
                   block_table=d.get("block_table"))

    @property
    def n_slices(self) -> int:
        return self.layers * self.seqs * self.kv_heads

    def c_struct(self) -> CCache:
        dt = DTYPE_BF16 if self.k.dtype == torch.bfloat16 else DTYPE_F32
        for t in (self.k, self.v, self.pos, self.lens):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("cache tensors must be contiguous CUDA tensors")
        if self.pos.dtype != torch.int32 or self.lens.dtype != torch.int32:
            raise ValueError("pos and lens must be int32")
        return CCache(self.layers, self.seqs, self.kv_heads, self.group, self.head_dim,
                      self.capacity, self.page_size, self.num_pages, self.max_pages_per_seq, dt,
                      self.k.data_ptr(), self.v.data_ptr(), self.pos.data_ptr(),
                      self.lens.data_ptr(),
                      None if self.block_table is None else self.block_table.data_ptr())


@dataclass
class Params:
    """Step parameters (nx_params). Budgets and forced counts are in decision units:
    rows at block_size 1, blocks of 32 rows at block_size 32."""
    budget: torch.Tensor           # int32 [seqs] on the device
    budget_max: int
    window: int
    walk_len: int = 3
    n_sink: int = 32
    n_recent: int = 32
    n_avg: int = 1
    mode: int = MODE_RESERVOIR
    lam: float = 0.5
    eps_tie: float = 1e-6
    seed: int = 0
    step: int = 0
    seq_id_base: int = 0
    layer_id_base: int = 0
    block_size: int = 1
    slice_budget: torch.Tensor | None = None   # int32 [slices] on the device (optional)

    def c_struct(self) -> CParams:
        if self.budget.dtype != torch.int32 or not self.budget.is_cuda:
            raise ValueError("budget must be an int32 CUDA tensor")
        sb = self.slice_budget
        if sb is not None and (sb.dtype != torch.int32 or not sb.is_cuda):
            raise ValueError("slice_budget must be an int32 CUDA tensor")
        return CParams(self.window, self.walk_len, self.n_sink, self.n_recent, self.n_avg,
                       self.mode, self.lam, self.eps_tie, self.budget.data_ptr(),
                       self.budget_max, self.seq_id_base, self.layer_id_base,
                       self.step & 0xFFFFFFFF, self.seed & 0xFFFFFFFFFFFFFFFF,
                       self.block_size, 0, None if sb is None else sb.data_ptr())


def _check(status: int, where: str):
    if status != NX_OK:
        raise NexusError(status, where)


def workspace_bytes(cache: Cache, params: Params) -> int:
    n = load().nexus_workspace_bytes(ctypes.byref(cache.c_struct()), ctypes.byref(params.c_struct()))
    if n == 0:
        raise NexusError(NX_ERR_INVALID_ARG, "nexus_workspace_bytes")
    return int(n)


def alloc_workspace(cache: Cache, params: Params) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks, above the 256 required
    return torch.empty(workspace_bytes(cache, params), dtype=torch.uint8, device=cache.k.device)


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def direct_scores(cache: Cache, q, params: Params, a_out, row_stats_out, ws, dev_status,
                  stream=None):
    _check(load().nexus_direct_scores(ctypes.byref(cache.c_struct()), _ptr(q),
                                      ctypes.byref(params.c_struct()), _ptr(a_out),
                                      _ptr(row_stats_out), _ptr(ws), ws.numel(),
                                      _ptr(dev_status), _stream(stream)),
           "nexus_direct_scores")


def walk(cache: Cache, q, params: Params, w_out, ctilde_out, ws, dev_status, stream=None):
    _check(load().nexus_walk(ctypes.byref(cache.c_struct()), _ptr(q),
                             ctypes.byref(params.c_struct()), _ptr(w_out), _ptr(ctilde_out),
                             _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream)),
           "nexus_walk")


def reservoir_select(w, cache: Cache, params: Params, keep_idx, ws, dev_status, stream=None):
    _check(load().nexus_reservoir_select(_ptr(w), ctypes.byref(cache.c_struct()),
                                         ctypes.byref(params.c_struct()), _ptr(keep_idx),
                                         _ptr(ws), ws.numel(), _ptr(dev_status),
                                         _stream(stream)),
           "nexus_reservoir_select")


def compact(cache: Cache, keep_idx, params: Params, ws, dev_status, stream=None):
    _check(load().kv_compact(ctypes.byref(cache.c_struct()), _ptr(keep_idx),
                             ctypes.byref(params.c_struct()), _ptr(ws), ws.numel(),
                             _ptr(dev_status), _stream(stream)),
           "kv_compact")


def evict_step(cache: Cache, q, params: Params, keep_idx_out, ws, dev_status, stream=None):
    _check(load().nexus_evict_step(ctypes.byref(cache.c_struct()), _ptr(q),
                                   ctypes.byref(params.c_struct()), _ptr(keep_idx_out),
                                   _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream)),
           "nexus_evict_step")


# ---------------------------------------------------------------------------
# Filling and reading the cache between two evictions
# ---------------------------------------------------------------------------

_PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


class Rotary:
    """Rotation frequencies as the library takes them: turns per position in units of 2^-64
    turn. freqs: radians per position of each rotated pair (head_dim / 2 of them or fewer;
    pairs are (i, i + len(freqs)), or (2i, 2i + 1) if interleaved)."""

    def __init__(self, freqs, interleaved: bool = False, device="cuda"):
        freqs = [float(f) for f in freqs]
        if not freqs or len(freqs) % 4 or not all(math.isfinite(f) for f in freqs):
            raise ValueError("freqs must be finite, a positive multiple of 4 of them")
        turns = [round(Fraction(f) / (2 * _PI) * (1 << 64)) & ((1 << 64) - 1) for f in freqs]
        self.table = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns],
                                  dtype=torch.int64, device=device)
        self.rotary_dim = 2 * len(freqs)
        self.interleaved = bool(interleaved)


@dataclass
class Image:
    """8-bit image of a bf16 cache (nx_image): k, v float8_e4m3fn in the cache's layout,
    float32 scales per block of rows, int32 rows [layers][seqs][kv_heads] held so far."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    rows: torch.Tensor

    def c_struct(self, cache: Cache) -> CImage:
        b = image_block(cache)
        n = cache.k.numel()
        blocks = n // cache.head_dim // b if cache.page_size else \
            cache.n_slices * (-(-cache.capacity // b))
        for t in (self.k, self.v, self.k_scale, self.v_scale, self.rows):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("image tensors must be contiguous CUDA tensors")
        if self.k.dtype != torch.float8_e4m3fn or self.v.dtype != torch.float8_e4m3fn:
            raise ValueError("image k and v must be float8_e4m3fn")
        if self.k_scale.dtype != torch.float32 or self.v_scale.dtype != torch.float32 or \
                self.rows.dtype != torch.int32:
            raise ValueError("image scales must be float32, rows int32")
        if self.k.numel() != n or self.v.numel() != n or self.rows.numel() != cache.n_slices or \
                self.k_scale.numel() != blocks or self.v_scale.numel() != blocks:
            raise ValueError("image sizes do not fit the cache")
        return CImage(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(),
                      self.v_scale.data_ptr(), self.rows.data_ptr())


def image_block(cache: Cache) -> int:
    """Rows that share a scale in an image of this cache."""
    return min(32, cache.page_size) if cache.page_size else 32


def new_image(cache: Cache) -> Image:
    """An image of the cache that holds no rows yet."""
    b = image_block(cache)
    if cache.page_size:
        blocks = (cache.layers, cache.num_pages, cache.kv_heads, cache.page_size // b)
    else:
        blocks = (cache.layers, cache.seqs, cache.kv_heads, -(-cache.capacity // b))
    dev = cache.k.device
    return Image(k=torch.zeros(cache.k.shape, dtype=torch.uint8, device=dev)
                 .view(torch.float8_e4m3fn),
                 v=torch.zeros(cache.v.shape, dtype=torch.uint8, device=dev)
                 .view(torch.float8_e4m3fn),
                 k_scale=torch.ones(blocks, device=dev), v_scale=torch.ones(blocks, device=dev),
                 rows=torch.zeros(cache.layers, cache.seqs, cache.kv_heads, dtype=torch.int32,
                                  device=dev))


def _tokens(cache: Cache, layer: int, tokens: int, max_tokens: int, cu_tokens) -> CTokens:
    if cu_tokens is not None:
        _int32(cu_tokens, cache.seqs + 1, "cu_tokens")
    return CTokens(layer, tokens, max_tokens, 0,
                   None if cu_tokens is None else cu_tokens.data_ptr())


def _int32(t, n: int, name: str):
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be {n} contiguous int32 values on the GPU")


def _status(t):
    if t is None or t.dtype != torch.int32 or not t.is_cuda:
        raise ValueError("dev_status must be an int32 tensor on the GPU")
    return ctypes.c_void_p(t.data_ptr())


def _heads(t, tokens: int, heads: int, cache: Cache, name: str):
    """A per-token tensor [tokens, heads, head_dim] whose heads lie behind one another;
    returns the elements between two tokens."""
    d = cache.head_dim
    if t.shape != (tokens, heads, d) or t.dtype != cache.k.dtype or not t.is_cuda:
        raise ValueError(f"{name} must be {(tokens, heads, d)} in the cache's type on the GPU")
    if not t.is_contiguous():
        step, head, one = t.stride()
        if one != 1 or (heads > 1 and head != d):
            raise ValueError(f"{name}: the heads of a token must lie behind one another")
        if tokens > 1:
            return step
    return heads * d


def append(cache: Cache, layer: int, q, k, v, token_pos, q_out, dev_status, *, max_tokens: int,
           cu_tokens=None, lens_in=None, rotary: Rotary | None = None, q_norm=None, k_norm=None,
           eps: float = 1e-6, image: Image | None = None, stream=None):
    """nexus_append: norms and rotates q and k, appends k, v and token_pos to the slices of
    `layer`, writes the queries to q_out. q [tokens, kv_heads * group, d] (or None, with
    q_out), k, v [tokens, kv_heads, d]: views of one packed projection will do. max_tokens:
    no sequence owns more tokens; cu_tokens int32 [seqs + 1], or None where each owns
    max_tokens. lens_in int32 [seqs, kv_heads]: rows to append behind, if not cache.lens (tokens
    behind it are taken back). image: an image of the cache forgets the blocks that held such
    tokens; without it the caller lowers image.rows, or attend reads their codes."""
    n, H = token_pos.numel(), cache.kv_heads
    HQ = H * cache.group
    _int32(token_pos, n, "token_pos")
    a = CAppend(k=k.data_ptr(), v=v.data_ptr(), pos=token_pos.data_ptr(), eps=eps)
    a.k_stride, a.v_stride = _heads(k, n, H, cache, "k"), _heads(v, n, H, cache, "v")
    if q is not None:
        a.q_stride, a.q = _heads(q, n, HQ, cache, "q"), q.data_ptr()
        if q_out is None or _heads(q_out, n, HQ, cache, "q_out") != HQ * cache.head_dim:
            raise ValueError("q_out must be packed")
        a.q_out = q_out.data_ptr()
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm go with q")
    if lens_in is not None:
        _int32(lens_in, cache.seqs * H, "lens_in")
        a.lens_in = lens_in.data_ptr()
    if rotary is not None:
        if not rotary.table.is_cuda:
            raise ValueError("the rotary table must be on the GPU")
        a.rotary, a.rotary_dim = rotary.table.data_ptr(), rotary.rotary_dim
        a.interleaved = rotary.interleaved
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None:
            if w.dtype != cache.k.dtype or not w.is_cuda or not w.is_contiguous() or \
                    w.numel() != cache.head_dim:
                raise ValueError(f"{name} must be head_dim values in the cache's type")
            setattr(a, name, w.data_ptr())
    im = None if image is None else ctypes.byref(image.c_struct(cache))
    _check(load().nexus_append_image(ctypes.byref(cache.c_struct()),
                                     ctypes.byref(_tokens(cache, layer, n, max_tokens, cu_tokens)),
                                     ctypes.byref(a), im, _status(dev_status), _stream(stream)),
           "nexus_append")


def quantize(cache: Cache, image: Image, dev_status, *, rows_in=None, stream=None):
    """nexus_quantize: brings the image up to date in every layer. rows_in int32 [layers,
    seqs, kv_heads]: rows that it holds already, if not image.rows (zeros behind an
    eviction, which moves rows)."""
    if rows_in is not None:
        _int32(rows_in, cache.n_slices, "rows_in")
    _check(load().nexus_quantize(ctypes.byref(cache.c_struct()),
                                 ctypes.byref(image.c_struct(cache)), _ptr(rows_in),
                                 _status(dev_status), _stream(stream)),
           "nexus_quantize")


def attend_workspace_bytes(cache: Cache, *, tokens: int, max_tokens: int) -> int:
    # the size goes by the bounds, not by how the tokens are dealt out: any non-null
    # cu_tokens will do
    t = CTokens(0, tokens, max_tokens, 0, cache.lens.data_ptr())
    n = load().nexus_attend_workspace_bytes(ctypes.byref(cache.c_struct()), ctypes.byref(t))
    if n == 0:
        raise NexusError(NX_ERR_INVALID_ARG, "nexus_attend_workspace_bytes")
    return int(n)


def alloc_attend_workspace(cache: Cache, *, tokens: int, max_tokens: int) -> torch.Tensor:
    return torch.empty(attend_workspace_bytes(cache, tokens=tokens, max_tokens=max_tokens),
                       dtype=torch.uint8, device=cache.k.device)


def attend(cache: Cache, layer: int, q, out, ws, dev_status, *, max_tokens: int, cu_tokens=None,
           causal: bool = True, scale: float | None = None, lse=None, image: Image | None = None,
           stream=None):
    """nexus_attend: softmax attention of q [tokens, kv_heads * group, d] over the slices of
    `layer`, into out (like q) and lse float32 [tokens, kv_heads * group] (optional). causal:
    the tokens are the slices' newest rows, and each sees what came before it and itself.
    scale: of the logits, 1 / sqrt(d) by default. image: read these 8-bit rows where held."""
    n, HQ = q.shape[0], cache.kv_heads * cache.group
    a = CAttend(q=q.data_ptr(), out=out.data_ptr(), causal=bool(causal),
                scale=cache.head_dim ** -0.5 if scale is None else scale)
    a.q_stride, a.out_stride = _heads(q, n, HQ, cache, "q"), _heads(out, n, HQ, cache, "out")
    if lse is not None:
        if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or \
                lse.numel() != n * HQ:
            raise ValueError("lse must be [tokens, kv_heads * group] float32 on the GPU")
        a.lse = lse.data_ptr()
    if not ws.is_cuda:
        raise ValueError("ws must be on the GPU")
    im = None if image is None else ctypes.byref(image.c_struct(cache))
    _check(load().nexus_attend(ctypes.byref(cache.c_struct()),
                               ctypes.byref(_tokens(cache, layer, n, max_tokens, cu_tokens)), im,
                               ctypes.byref(a), _ptr(ws), ws.numel(), _status(dev_status),
                               _stream(stream)),
           "nexus_attend")
