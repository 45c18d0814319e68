"""GB300-native MiniMax Sparse Attention (MSA) layer: Python binding of libmsa_gb300.so.

Each function marshals torch CUDA tensors into the C ABI of ``include/msa.h`` (pointers,
sizes, the current CUDA stream) and calls it; every step of the computation runs in the
library's CUDA kernels. There is no CPU or PyTorch fallback: a missing library raises.

Stage 1  ``index_score_topk``        block scores + top-k selection per (query row, KV group)
         ``build_sparse_page_table`` flattened per-(row, group) page tables over the
                                     strided per-head KV view
Stage 2  ``paged_sparse_decode``     paged decode attention over the selected pages
         ``sparse_prefill``          KV-block-major prefill attention + LSE merge
Serving  ``build_page_tables``       page tables, lengths and slot maps from request lengths
batch    ``append_kv``               new tokens into the paged caches
         ``shared_prefix_decode``    dense paged decode for requests that share a prefix
         ``chunk_attention``         causal attention of a ragged batch of new tokens, paged
Quantised ``append_kv_fp8``          new tokens quantised into e4m3 caches
cache    ``gather_kv_fp8``           rows of them read back as bf16
         ``paged_sparse_decode_fp8`` paged sparse decode on them
Pieces   ``prefill_bucket``, ``lse_merge``, ``device_error``
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import MSAError, library_path, load

__all__ = ["index_score_topk", "index_score_topk_noalloc", "build_sparse_page_table", "paged_sparse_decode", "sparse_prefill",
           "build_page_tables", "append_kv", "shared_prefix_decode", "chunk_attention",
           "append_kv_fp8", "gather_kv_fp8", "paged_sparse_decode_fp8",
           "prefill_bucket", "lse_merge", "device_error", "Workspace", "MSAError", "load",
           "library_path", "BLOCK"]

BLOCK = 128


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {tuple(t.shape)}")
    return t


class Workspace:
    """Caller-owned scratch memory for the C ABI, grown on demand and reused.

    One Workspace serves every call made on one stream; calls that may overlap on the
    GPU need separate Workspace objects.
    """

    def __init__(self):
        self._bufs: dict = {}

    def get(self, key: str, nbytes: int, device, zero: bool = False) -> torch.Tensor:
        nbytes = max(int(nbytes), 256)
        cur = self._bufs.get(key)
        if cur is None or cur.numel() < nbytes or cur.device != torch.device(device):
            alloc = torch.zeros if zero else torch.empty
            cur = alloc(nbytes, dtype=torch.uint8, device=device)
            self._bufs[key] = cur
        return cur


_default_ws: dict = {}


def _ws(ws: Workspace | None, device) -> Workspace:
    if ws is not None:
        return ws
    key = (torch.device(device), torch.cuda.current_stream(device).cuda_stream)
    if key not in _default_ws:
        _default_ws[key] = Workspace()
    return _default_ws[key]


# ------------------------------------------------------------------------------ stage 1

def index_score_topk(q_idx, k_idx_pages, page_table, seq_lens, N: int, topk: int,
                     with_scores: bool = True, workspace: Workspace | None = None,
                     out=None):
    """Block scores and top-k selection (``msa_index_score_topk``).

    q_idx [B*N, Hkv, Di] bf16, k_idx_pages [P, 128, Hkv, Di] bf16, page_table [B, max_blocks]
    int32, seq_lens [B] int32. Returns (block_ids [B*N, Hkv, topk] int32,
    scores [B*N, Hkv, topk] fp32 or None).
    """
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    _need(k_idx_pages, "k_idx_pages", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, max_blocks = page_table.shape
    R, Hkv, Di = q_idx.shape
    if R != B * N or k_idx_pages.shape[1:] != (BLOCK, Hkv, Di) or seq_lens.numel() != B:
        raise ValueError("index_score_topk: inconsistent shapes")
    dev = q_idx.device
    if out is None:
        ids = torch.empty((R, Hkv, topk), dtype=torch.int32, device=dev)
        sc = torch.empty((R, Hkv, topk), dtype=torch.float32, device=dev) if with_scores else None
    else:
        ids, sc = out
    lib = load()
    nbytes = lib.msa_index_score_topk_workspace_size(B, N, Hkv, max_blocks)
    buf = _ws(workspace, dev).get("score", nbytes, dev)
    rc = lib.msa_index_score_topk(_ptr(q_idx), _ptr(k_idx_pages), _ptr(page_table), _ptr(seq_lens),
                                  B, N, Hkv, Di, max_blocks, k_idx_pages.shape[0], topk, _ptr(ids),
                                  _ptr(sc), _ptr(buf), buf.numel(), _stream(dev))
    _lib.check("msa_index_score_topk", rc)
    return ids, sc


def index_score_topk_page_table(q_idx, k_idx_pages, page_table, seq_lens, N: int, topk: int,
                                with_scores: bool = True, workspace: Workspace | None = None):
    """Selection and its sparse page table in one call (``msa_index_score_topk_page_table``).

    Arguments as ``index_score_topk``. Returns (block_ids [B*N, Hkv, topk] int32, scores or None,
    flat_page_table [B*N*Hkv, topk] int32, flat_kv_lens [B*N*Hkv] int32).
    """
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    _need(k_idx_pages, "k_idx_pages", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, max_blocks = page_table.shape
    R, Hkv, Di = q_idx.shape
    if R != B * N or k_idx_pages.shape[1:] != (BLOCK, Hkv, Di) or seq_lens.numel() != B:
        raise ValueError("index_score_topk_page_table: inconsistent shapes")
    dev = q_idx.device
    ids = torch.empty((R, Hkv, topk), dtype=torch.int32, device=dev)
    sc = torch.empty((R, Hkv, topk), dtype=torch.float32, device=dev) if with_scores else None
    fpt = torch.empty((R * Hkv, topk), dtype=torch.int32, device=dev)
    lens = torch.empty((R * Hkv,), dtype=torch.int32, device=dev)
    lib = load()
    nbytes = lib.msa_index_score_topk_workspace_size(B, N, Hkv, max_blocks)
    buf = _ws(workspace, dev).get("score", nbytes, dev)
    rc = lib.msa_index_score_topk_page_table(
        _ptr(q_idx), _ptr(k_idx_pages), _ptr(page_table), _ptr(seq_lens), B, N, Hkv, Di,
        max_blocks, k_idx_pages.shape[0], topk, _ptr(ids), _ptr(sc), _ptr(fpt), _ptr(lens),
        _ptr(buf), buf.numel(), _stream(dev))
    _lib.check("msa_index_score_topk_page_table", rc)
    return ids, sc, fpt, lens


def index_score_topk_noalloc(q_idx, k_idx_pages, page_table, seq_lens, N: int, topk: int,
                             with_scores: bool = True, out=None):
    """``index_score_topk`` without a workspace (``msa_index_score_topk_noalloc``).

    For callers that cannot hand the library device scratch memory: the library uses a
    fixed 8 MiB array of its own on each device instead. Calls on one device share that
    array, so calls that may overlap on the GPU must not use this function. The first
    call on a device resolves the array's address; make it before any stream capture.
    Raises MSAError (MSA_ERR_UNSUPPORTED) when B*N*Hkv*max_blocks needs more scratch.
    """
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    _need(k_idx_pages, "k_idx_pages", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, max_blocks = page_table.shape
    R, Hkv, Di = q_idx.shape
    if R != B * N or k_idx_pages.shape[1:] != (BLOCK, Hkv, Di) or seq_lens.numel() != B:
        raise ValueError("index_score_topk_noalloc: inconsistent shapes")
    dev = q_idx.device
    if out is None:
        ids = torch.empty((R, Hkv, topk), dtype=torch.int32, device=dev)
        sc = torch.empty((R, Hkv, topk), dtype=torch.float32, device=dev) if with_scores else None
    else:
        ids, sc = out
    rc = load().msa_index_score_topk_noalloc(_ptr(q_idx), _ptr(k_idx_pages), _ptr(page_table),
                                             _ptr(seq_lens), B, N, Hkv, Di, max_blocks,
                                             k_idx_pages.shape[0], topk, _ptr(ids), _ptr(sc),
                                             _stream(dev))
    _lib.check("msa_index_score_topk_noalloc", rc)
    return ids, sc


def build_sparse_page_table(block_ids, page_table, seq_lens, N: int, num_pages: int, out=None):
    """Flattened sparse page tables (``msa_build_sparse_page_table``).

    Returns (flat_page_table [B*N*Hkv, topk] int32, flat_kv_lens [B*N*Hkv] int32).
    """
    _need(block_ids, "block_ids", torch.int32, 3)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    R, Hkv, topk = block_ids.shape
    B, max_blocks = page_table.shape
    if R != B * N:
        raise ValueError("build_sparse_page_table: block_ids rows != B*N")
    dev = block_ids.device
    if out is None:
        fpt = torch.empty((R * Hkv, topk), dtype=torch.int32, device=dev)
        lens = torch.empty((R * Hkv,), dtype=torch.int32, device=dev)
    else:
        fpt, lens = out
    rc = load().msa_build_sparse_page_table(_ptr(block_ids), _ptr(page_table), _ptr(seq_lens), B, N,
                                            Hkv, topk, max_blocks, num_pages, _ptr(fpt), _ptr(lens),
                                            _stream(dev))
    _lib.check("msa_build_sparse_page_table", rc)
    return fpt, lens


# ------------------------------------------------------------------------------ stage 2

def stage_selected_kv(k_cache, v_cache, flat_page_table, out=None):
    """Copy the selected blocks' K/V to a device staging cache (``msa_stage_selected_kv``).

    k_cache, v_cache [P, 128, Hkv, D] bf16: CUDA tensors or pinned host tensors (read by the
    device directly); flat_page_table [R*Hkv, topk] int32 (CUDA). Returns (k_stage, v_stage
    [R*topk, 128, Hkv, D] bf16, stage_page_table [R*Hkv, topk] int32) for ``paged_sparse_decode``,
    written into ``out`` when given.
    """
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{name}: must be a CUDA tensor or pinned host memory")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous bf16 [P, 128, Hkv, D] tensor")
    _need(flat_page_table, "flat_page_table", torch.int32, 2)
    P, _, Hkv, D = k_cache.shape
    RH, topk = flat_page_table.shape
    if v_cache.shape != k_cache.shape or RH % Hkv:
        raise ValueError("stage_selected_kv: inconsistent shapes")
    R = RH // Hkv
    dev = flat_page_table.device
    if out is None:
        k_stage = torch.empty((R * topk, BLOCK, Hkv, D), dtype=torch.bfloat16, device=dev)
        v_stage = torch.empty_like(k_stage)
        spt = torch.empty_like(flat_page_table)
    else:
        k_stage, v_stage, spt = out
        _need(k_stage, "k_stage", torch.bfloat16, 4)
        _need(v_stage, "v_stage", torch.bfloat16, 4)
        _need(spt, "stage_page_table", torch.int32, 2)
        if (k_stage.shape != (R * topk, BLOCK, Hkv, D) or v_stage.shape != k_stage.shape
                or spt.shape != flat_page_table.shape):
            raise ValueError("stage_selected_kv: output shapes do not match")
    rc = load().msa_stage_selected_kv(k_cache.data_ptr(), v_cache.data_ptr(), P,
                                      _ptr(flat_page_table), R, Hkv, D, topk, _ptr(k_stage),
                                      _ptr(v_stage), _ptr(spt), _stream(dev))
    _lib.check("msa_stage_selected_kv", rc)
    return k_stage, v_stage, spt


def paged_sparse_decode(q, k_cache, v_cache, flat_page_table, flat_kv_lens,
                        with_lse: bool = True, workspace: Workspace | None = None, out=None):
    """Paged sparse decode attention (``msa_paged_sparse_decode``).

    q [R, Hq, D] bf16; caches [P, 128, Hkv, D] bf16; flat tables from
    ``build_sparse_page_table``. Returns (o [R, Hq, D] bf16, lse [R, Hq] fp32 or None).
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(flat_page_table, "flat_page_table", torch.int32, 2)
    _need(flat_kv_lens, "flat_kv_lens", torch.int32, 1)
    R, Hq, D = q.shape
    P, _, Hkv, _ = k_cache.shape
    topk = flat_page_table.shape[1]
    if v_cache.shape != k_cache.shape or flat_page_table.shape[0] != R * Hkv:
        raise ValueError("paged_sparse_decode: inconsistent shapes")
    dev = q.device
    if out is None:
        o = torch.empty((R, Hq, D), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((R, Hq), dtype=torch.float32, device=dev) if with_lse else None
    else:
        o, lse = out
    lib = load()
    nbytes = lib.msa_paged_sparse_decode_workspace_size(R, Hq, Hkv, topk)
    buf = _ws(workspace, dev).get("decode", nbytes, dev)
    rc = lib.msa_paged_sparse_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(flat_page_table),
                                     _ptr(flat_kv_lens), R, Hq, Hkv, D, topk, P, _ptr(o), _ptr(lse),
                                     _ptr(buf), buf.numel(), _stream(dev))
    _lib.check("msa_paged_sparse_decode", rc)
    return o, lse


def sparse_prefill(q, k, v, block_ids, with_lse: bool = True,
                   workspace: Workspace | None = None, out=None):
    """KV-block-major sparse prefill with LSE merge (``msa_sparse_prefill``).

    q [T, Hq, D] bf16 at positions S_kv-T..S_kv-1; k, v [S_kv, Hkv, D] bf16;
    block_ids [T, Hkv, topk] int32. Returns (o [T, Hq, D] bf16, lse [T, Hq] fp32 or None).
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(block_ids, "block_ids", torch.int32, 3)
    T, Hq, D = q.shape
    S_kv, Hkv, _ = k.shape
    topk = block_ids.shape[2]
    if v.shape != k.shape or block_ids.shape[:2] != (T, Hkv):
        raise ValueError("sparse_prefill: inconsistent shapes")
    dev = q.device
    if out is None:
        o = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if with_lse else None
    else:
        o, lse = out
    lib = load()
    nbytes = lib.msa_sparse_prefill_workspace_size(T, S_kv, Hq, Hkv, topk)
    buf = _ws(workspace, dev).get("prefill", nbytes, dev)
    rc = lib.msa_sparse_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(block_ids), T, S_kv, Hq, Hkv, D, topk,
                                _ptr(o), _ptr(lse), _ptr(buf), buf.numel(), _stream(dev))
    _lib.check("msa_sparse_prefill", rc)
    return o, lse


def sparse_prefill_paged(q, k_cache, v_cache, page_table, block_ids, S_kv: int,
                         with_lse: bool = True, workspace: Workspace | None = None, out=None):
    """Sparse prefill over a paged K/V cache (``msa_sparse_prefill_paged``).

    q [T, Hq, D] bf16 at positions S_kv-T..S_kv-1; k_cache, v_cache [P, 128, Hkv, D] bf16;
    page_table [ceil(S_kv/128)] int32 (page of each 128-token block); block_ids
    [T, Hkv, topk] int32. Returns (o [T, Hq, D] bf16, lse [T, Hq] fp32 or None).
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 1)
    _need(block_ids, "block_ids", torch.int32, 3)
    T, Hq, D = q.shape
    P, _, Hkv, _ = k_cache.shape
    topk = block_ids.shape[2]
    if v_cache.shape != k_cache.shape or block_ids.shape[:2] != (T, Hkv) \
            or page_table.numel() < (S_kv + 127) // 128:
        raise ValueError("sparse_prefill_paged: inconsistent shapes")
    dev = q.device
    if out is None:
        o = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if with_lse else None
    else:
        o, lse = out
    lib = load()
    nbytes = lib.msa_sparse_prefill_workspace_size(T, S_kv, Hq, Hkv, topk)
    buf = _ws(workspace, dev).get("prefill", nbytes, dev)
    rc = lib.msa_sparse_prefill_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), P,
                                      _ptr(block_ids), T, S_kv, Hq, Hkv, D, topk, _ptr(o),
                                      _ptr(lse), _ptr(buf), buf.numel(), _stream(dev))
    _lib.check("msa_sparse_prefill_paged", rc)
    return o, lse


# ------------------------------------------------------------------------------ serving batch
#
# These calls sit in a decode loop next to kernels of a few microseconds, so their host side is
# kept short: one pass of attribute tests per tensor, no device guard when the device is current.
# Measured per eager call whose kernels are shorter: append 10 to 12 us (22 with the other calls'
# checks), page tables 21 to 25 us (30; five outputs to allocate), shared-prefix decode 25 to 29 us
# (two launches, eleven tensor maps).

def _check(name: str, t, dtype, ndim: int, dev):
    """A contiguous CUDA tensor of that type and rank on `dev`; the errors of ``_need``."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()
            and t.device == dev):
        _need(t, name, dtype, ndim)
        raise ValueError(f"{name}: on {t.device}, expected {dev}")


def _sizes(name: str, *sizes: int):
    """Sizes become int32 arguments, which would wrap around without an error."""
    if max(sizes) > 2 ** 31 - 1:
        raise ValueError(f"{name}: a size of {max(sizes)} exceeds int32")


def _call(dev, fn, *args):
    """fn(*args, current stream of `dev`) with `dev` current."""
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch.cuda.current_device() == dev.index:
        return fn(*args, stream)
    with torch.cuda.device(dev):
        return fn(*args, stream)


def _scratch_call(dev, workspace: Workspace | None, key: str, size, fn):
    """fn(pointer, bytes, stream) with `dev` current and size() bytes of scratch, from `workspace` or, for
    this call alone, from the caching allocator: in the stream's order, as a tensor's memory would be, but
    without the tensor. (A call of one row on 2048 keys takes the host 19.2 us so, 23.3 with a tensor, 22.1
    with the allocator's calls in torch.cuda.)"""
    def run(stream):
        nbytes = max(256, size())
        if workspace is not None:
            buf = workspace.get(key, nbytes, dev)
            return fn(buf.data_ptr(), buf.numel(), stream)
        ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, stream)
        try:
            return fn(ptr, nbytes, stream)
        finally:
            torch._C._cuda_cudaCachingAllocator_raw_delete(ptr)

    return _call(dev, run)


def build_page_tables(prev_lens, new_lens, page_table, free_pages, pages_used, T: int,
                      num_pages: int, shared_pages=None, out=None):
    """Page tables, lengths and slot maps of a step, from lengths (``msa_build_page_tables``).

    prev_lens, new_lens [B] int32 (tokens held, tokens added); page_table [B, max_blocks] int32,
    updated in place; free_pages [F] int32, taken in order from index pages_used [1] int32 on;
    T token rows (those behind the last token get -1); shared_pages [n] int32: a cached prefix's
    whole pages, entered for every request that holds at least n*128 tokens, whatever its table
    held: only for a batch whose long requests are all behind that prefix. Returns (seq_lens
    [B], cu_tokens [B+1], slot_map [T], positions [T], pages_used [1]), all int32, written into
    ``out`` when given (no output may overlap an input or another output).
    """
    i32 = torch.int32
    _sizes("build_page_tables", T, num_pages)
    _need(page_table, "page_table", i32, 2)
    dev = page_table.device
    _check("prev_lens", prev_lens, i32, 1, dev)
    _check("new_lens", new_lens, i32, 1, dev)
    _check("free_pages", free_pages, i32, 1, dev)
    _check("pages_used", pages_used, i32, 1, dev)
    B, max_blocks = page_table.shape
    shared, num_shared = None, 0
    if shared_pages is not None:
        _check("shared_pages", shared_pages, i32, 1, dev)
        shared, num_shared = shared_pages.data_ptr(), shared_pages.numel()
    if prev_lens.numel() != B or new_lens.numel() != B or pages_used.numel() != 1 or T < 0:
        raise ValueError("build_page_tables: inconsistent shapes")
    _sizes("build_page_tables", B, max_blocks, free_pages.numel(), num_shared)
    sizes = (B, B + 1, T, T, 1)
    if out is None:
        out = [torch.empty(n, dtype=i32, device=dev) for n in sizes]
    else:
        for name, t, n in zip(("seq_lens", "cu_tokens", "slot_map", "positions", "pages_used"), out,
                              sizes, strict=True):
            _check(f"out {name}", t, i32, 1, dev)
            if t.numel() != n:
                raise ValueError(f"build_page_tables: out {name} has {t.numel()} elements, expected {n}")
    seq_lens, cu_tokens, slot_map, positions, used_out = out
    rc = _call(dev, load().msa_build_page_tables, prev_lens.data_ptr(), new_lens.data_ptr(), B, max_blocks,
               page_table.data_ptr(), free_pages.data_ptr(), free_pages.numel(), pages_used.data_ptr(),
               shared, num_shared, num_pages, T, seq_lens.data_ptr(), cu_tokens.data_ptr(),
               slot_map.data_ptr(), positions.data_ptr(), used_out.data_ptr())
    _lib.check("msa_build_page_tables", rc)
    return seq_lens, cu_tokens, slot_map, positions, used_out


def _need_rows(t, name: str, T: int, Hkv: int, d: int, dev):
    """A [T, Hkv, d] bf16 tensor whose token rows are dense; returns (pointer, row stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {torch.bfloat16}")
    if t.shape != (T, Hkv, d):
        raise ValueError(f"{name}: expected shape {(T, Hkv, d)}, got {tuple(t.shape)}")
    stride = t.stride()
    if T and (stride[2] != 1 or (Hkv > 1 and stride[1] != d)):
        raise ValueError(f"{name}: the heads of a token row must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")
    return t.data_ptr(), stride[0] if T > 1 else Hkv * d


def append_kv(k, v, k_idx, slot_map, k_cache, v_cache, k_idx_pages):
    """Write new tokens into the paged caches, in place (``msa_append_kv``).

    k, v [T, Hkv, D] and k_idx [T, Hkv, Di] bf16, token rows dense but their stride free (slices
    of a fused projection; 16-byte aligned, a multiple of 8 elements); slot_map [T] int32 from
    ``build_page_tables`` (negative: skipped; non-negative slots must differ, and no cell written
    may be a row read); k_cache, v_cache [P, 128, Hkv, D], k_idx_pages [P, 128, Hkv, Di] bf16. k, v
    and their caches, or k_idx and its pages, may be None.
    """
    if (k is None) != (v is None) or (k is None) != (k_cache is None) or \
            (k is None) != (v_cache is None) or (k_idx is None) != (k_idx_pages is None) or \
            (k is None and k_idx is None):
        raise ValueError("append_kv: k, v and their caches, or k_idx and its pages, come together")
    _need(slot_map, "slot_map", torch.int32, 1)
    dev = slot_map.device
    T = slot_map.numel()
    _sizes("append_kv", T)
    kp = vp = xp = kc = vc = xc = None
    ks = vs = xs = 0
    D = Di = BLOCK
    P, page, Hkv = (k_cache if k is not None else k_idx_pages).shape[:3]
    if page != BLOCK:
        raise ValueError("append_kv: caches must have 128-token pages")
    if k is not None:
        _check("k_cache", k_cache, torch.bfloat16, 4, dev)
        _check("v_cache", v_cache, torch.bfloat16, 4, dev)
        D = k_cache.shape[3]
        if v_cache.shape != k_cache.shape:
            raise ValueError("append_kv: inconsistent shapes")
        kp, ks = _need_rows(k, "k", T, Hkv, D, dev)
        vp, vs = _need_rows(v, "v", T, Hkv, D, dev)
        kc, vc = k_cache.data_ptr(), v_cache.data_ptr()
    if k_idx is not None:
        _check("k_idx_pages", k_idx_pages, torch.bfloat16, 4, dev)
        Di = k_idx_pages.shape[3]
        if k_idx_pages.shape[:3] != (P, page, Hkv):
            raise ValueError("append_kv: inconsistent shapes")
        xp, xs = _need_rows(k_idx, "k_idx", T, Hkv, Di, dev)
        xc = k_idx_pages.data_ptr()
    rc = _call(dev, load().msa_append_kv, kp, ks, vp, vs, xp, xs, slot_map.data_ptr(), T, Hkv, D, Di, P,
               kc, vc, xc)
    _lib.check("msa_append_kv", rc)


def shared_prefix_decode(q, k_cache, v_cache, page_table, seq_lens, shared_len, N: int = 1,
                         with_lse: bool = True, workspace: Workspace | None = None, out=None):
    """Dense paged decode for requests that share a prefix (``msa_shared_prefix_decode``).

    q [B*N, Hq, D] bf16 (the last N positions of each request); caches [P, 128, Hkv, D] bf16;
    page_table [B, max_blocks] int32; seq_lens [B] int32 (0: a padding request); shared_len [1]
    int32: leading tokens that hold the same keys and values for every request; of these the whole
    64-token steps that every active request's rows see are read once, so a single short request
    costs the batch its sharing. Returns
    (o [B*N, Hq, D] bf16, lse [B*N, Hq] fp32 or None), written into ``out`` when given. Sums and
    lse are fp32; the softmax weights are rounded to bf16 for their product with V, as in the
    library's other attention calls (relative RMS error of o on random values: 2.3e-3, against
    1.7e-3 for weights in fp32). Without ``workspace`` the scratch comes from the caching allocator
    for this call alone, so captured graphs and other streams do not share it (59 MB for B 256, N 1,
    Hq 64, Hkv 8, 0.9 GB for B 4096: see ``msa_shared_prefix_decode_workspace_size``).
    """
    bf16, i32 = torch.bfloat16, torch.int32
    _need(q, "q", bf16, 3)
    dev = q.device
    _check("k_cache", k_cache, bf16, 4, dev)
    _check("v_cache", v_cache, bf16, 4, dev)
    _check("page_table", page_table, i32, 2, dev)
    _check("seq_lens", seq_lens, i32, 1, dev)
    _check("shared_len", shared_len, i32, 1, dev)
    R, Hq, D = q.shape
    P, page, Hkv, Dk = k_cache.shape
    B, max_blocks = page_table.shape
    if R != B * N or v_cache.shape != k_cache.shape or Dk != D or page != BLOCK \
            or seq_lens.numel() != B or shared_len.numel() != 1:
        raise ValueError("shared_prefix_decode: inconsistent shapes")
    _sizes("shared_prefix_decode", B, N, Hq, max_blocks)
    if out is None:
        o = torch.empty((R, Hq, D), dtype=bf16, device=dev)
        lse = torch.empty((R, Hq), dtype=torch.float32, device=dev) if with_lse else None
    else:
        o, lse = out
        _check("out o", o, bf16, 3, dev)
        if lse is not None:
            _check("out lse", lse, torch.float32, 2, dev)
        if o.shape != q.shape or (lse is not None and lse.shape != (R, Hq)):
            raise ValueError("shared_prefix_decode: output shapes do not match")
    lib = load()

    def run(stream):
        # on the device: the size goes with its SM count
        nbytes = max(256, lib.msa_shared_prefix_decode_workspace_size(B, N, Hq, Hkv))
        buf = torch.empty(nbytes, dtype=torch.uint8, device=dev) if workspace is None \
            else workspace.get("shared_prefix", nbytes, dev)
        return lib.msa_shared_prefix_decode(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
            seq_lens.data_ptr(), shared_len.data_ptr(), B, N, Hq, Hkv, D, max_blocks, P, o.data_ptr(),
            None if lse is None else lse.data_ptr(), buf.data_ptr(), nbytes if workspace is None
            else buf.numel(), stream)

    _lib.check("msa_shared_prefix_decode", _call(dev, run))
    return o, lse


def chunk_attention(q, k_cache, v_cache, page_table, seq_lens, cu_tokens, with_lse: bool = True,
                    workspace: Workspace | None = None, out=None):
    """Causal attention of a ragged batch of new tokens over the paged cache (``msa_chunk_attention``).

    q [T, Hq, D] bf16, token rows dense but their stride free (a slice of a fused projection; 16-byte
    aligned, a multiple of 8 elements); caches [P, 128, Hkv, D] bf16; page_table [B, max_blocks],
    seq_lens [B], cu_tokens [B+1] int32, as ``build_page_tables`` leaves them: request b's new tokens,
    any number of them, are rows cu_tokens[b]..cu_tokens[b+1]-1, at its last positions, and see every
    key up to their own (prompts, chunks and decode rows in one call). Returns (o [T, Hq, D] bf16,
    lse [T, Hq] fp32 or None), written into ``out`` when given; rows behind cu_tokens[B] are left as
    they were (undefined without ``out``). Without ``workspace`` the scratch comes from the caching
    allocator for this call alone, so captured graphs and other streams do not share it (0.30 GB for
    2048 rows on 485 blocks: see ``msa_chunk_attention_workspace_size``).
    """
    bf16, i32 = torch.bfloat16, torch.int32
    _need(k_cache, "k_cache", bf16, 4)
    dev = k_cache.device
    _check("v_cache", v_cache, bf16, 4, dev)
    _check("page_table", page_table, i32, 2, dev)
    _check("seq_lens", seq_lens, i32, 1, dev)
    _check("cu_tokens", cu_tokens, i32, 1, dev)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q: expected a [T, Hq, D] tensor")
    T, Hq, D = q.shape
    qp, q_stride = _need_rows(q, "q", T, Hq, D, dev)
    P, page, Hkv, Dk = k_cache.shape
    B, max_blocks = page_table.shape
    if v_cache.shape != k_cache.shape or Dk != D or page != BLOCK or seq_lens.numel() != B \
            or cu_tokens.numel() != B + 1:
        raise ValueError("chunk_attention: inconsistent shapes")
    _sizes("chunk_attention", B, T, Hq, max_blocks)
    if out is None:
        o = torch.empty((T, Hq, D), dtype=bf16, device=dev)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if with_lse else None
    else:
        o, lse = out
        _check("out o", o, bf16, 3, dev)
        if lse is not None:
            _check("out lse", lse, torch.float32, 2, dev)
        if o.shape != q.shape or (lse is not None and lse.shape != (T, Hq)):
            raise ValueError("chunk_attention: output shapes do not match")
    lib = load()
    rc = _scratch_call(  # the size goes with the device's SM count
        dev, workspace, "chunk", lambda: lib.msa_chunk_attention_workspace_size(B, T, Hq, Hkv, max_blocks),
        lambda ws, nbytes, stream: lib.msa_chunk_attention(
            qp, q_stride, k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
            cu_tokens.data_ptr(), B, T, Hq, Hkv, D, max_blocks, P, o.data_ptr(),
            None if lse is None else lse.data_ptr(), ws, nbytes, stream))
    _lib.check("msa_chunk_attention", rc)
    return o, lse


# ------------------------------------------------------------------------------ quantised cache

def _fp8_caches(k_cache, v_cache, k_scale, v_scale):
    """Checks e4m3 caches [P, Hkv, 128, D] and their uint8 scales [P, Hkv, 128]; returns (P, Hkv, D, device)."""
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    _need(k_cache, "k_cache", f8, 4)
    dev = k_cache.device
    _check("v_cache", v_cache, f8, 4, dev)
    _check("k_scale", k_scale, u8, 3, dev)
    _check("v_scale", v_scale, u8, 3, dev)
    P, Hkv, page, D = k_cache.shape
    if page != BLOCK or v_cache.shape != k_cache.shape or k_scale.shape != (P, Hkv, page) \
            or v_scale.shape != (P, Hkv, page):
        raise ValueError("quantised caches: expected [P, Hkv, 128, D] and scales [P, Hkv, 128]")
    _sizes("quantised caches", P, Hkv, D)
    return P, Hkv, D, dev


def append_kv_fp8(k, v, slot_map, k_cache, v_cache, k_scale, v_scale):
    """Quantise new tokens into e4m3 caches, in place (``msa_append_kv_fp8``).

    k, v [T, Hkv, D] bf16, token rows dense but their stride free, as in ``append_kv``; slot_map [T]
    int32 (negative: skipped; non-negative slots must differ); k_cache, v_cache [P, Hkv, 128, D]
    float8_e4m3fn; k_scale, v_scale [P, Hkv, 128] uint8. A row (one token, one group) is held as e4m3
    numbers times 2^(scale - 127), the smallest power of two that brings its largest magnitude to
    at most 448; each value is then off by at most 2^-4 of itself (2^-10 of that power near zero).
    The key index goes through ``append_kv``, which takes k and v of None.
    """
    P, Hkv, D, dev = _fp8_caches(k_cache, v_cache, k_scale, v_scale)
    _check("slot_map", slot_map, torch.int32, 1, dev)
    T = slot_map.numel()
    _sizes("append_kv_fp8", T)
    kp, ks = _need_rows(k, "k", T, Hkv, D, dev)
    vp, vs = _need_rows(v, "v", T, Hkv, D, dev)
    rc = _call(dev, load().msa_append_kv_fp8, kp, ks, vp, vs, slot_map.data_ptr(), T, Hkv, D, P,
               k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())
    _lib.check("msa_append_kv_fp8", rc)


def gather_kv_fp8(k_cache, v_cache, k_scale, v_scale, slots, out=None):
    """Rows of e4m3 caches read back as bf16 (``msa_gather_kv_fp8``).

    Caches as in ``append_kv_fp8``; slots [T] int32 (page*128 + offset; negative: the row is left as it
    was, undefined without ``out``). Returns (k, v) [T, Hkv, D] bf16, the values that the caches hold,
    exactly; written into ``out`` when given.
    """
    P, Hkv, D, dev = _fp8_caches(k_cache, v_cache, k_scale, v_scale)
    _check("slots", slots, torch.int32, 1, dev)
    T = slots.numel()
    _sizes("gather_kv_fp8", T)
    if out is None:
        k = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=dev)
        v = torch.empty_like(k)
    else:
        k, v = out
        for name, t in (("out k", k), ("out v", v)):
            _check(name, t, torch.bfloat16, 3, dev)
            if t.shape != (T, Hkv, D):
                raise ValueError(f"gather_kv_fp8: {name} has shape {tuple(t.shape)}, expected {(T, Hkv, D)}")
    rc = _call(dev, load().msa_gather_kv_fp8, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
               v_scale.data_ptr(), P, slots.data_ptr(), T, Hkv, D, k.data_ptr(), v.data_ptr())
    _lib.check("msa_gather_kv_fp8", rc)
    return k, v


def paged_sparse_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, flat_page_table, flat_kv_lens,
                            with_lse: bool = True, workspace: Workspace | None = None, out=None):
    """Paged sparse decode attention on e4m3 caches (``msa_paged_sparse_decode_fp8``).

    q [R, Hq, D] bf16; caches as in ``append_kv_fp8``; flat tables from ``build_sparse_page_table``, the
    same as for ``paged_sparse_decode``. Returns (o [R, Hq, D] bf16, lse [R, Hq] fp32 or None): attention
    on the values that the caches hold, written into ``out`` when given. Without ``workspace`` the
    scratch comes from the caching allocator for this call alone.
    """
    bf16, i32 = torch.bfloat16, torch.int32
    P, Hkv, Dk, dev = _fp8_caches(k_cache, v_cache, k_scale, v_scale)
    _check("q", q, bf16, 3, dev)
    _check("flat_page_table", flat_page_table, i32, 2, dev)
    _check("flat_kv_lens", flat_kv_lens, i32, 1, dev)
    R, Hq, D = q.shape
    topk = flat_page_table.shape[1]
    if D != Dk or flat_page_table.shape[0] != R * Hkv or flat_kv_lens.numel() != R * Hkv:
        raise ValueError("paged_sparse_decode_fp8: inconsistent shapes")
    _sizes("paged_sparse_decode_fp8", R, Hq, topk)
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((R, Hq), dtype=torch.float32, device=dev) if with_lse else None
    else:
        o, lse = out
        _check("out o", o, bf16, 3, dev)
        if lse is not None:
            _check("out lse", lse, torch.float32, 2, dev)
        if o.shape != q.shape or (lse is not None and lse.shape != (R, Hq)):
            raise ValueError("paged_sparse_decode_fp8: output shapes do not match")
    lib = load()
    rc = _scratch_call(
        dev, workspace, "decode_fp8", lambda: lib.msa_paged_sparse_decode_workspace_size(R, Hq, Hkv, topk),
        lambda ws, nbytes, stream: lib.msa_paged_sparse_decode_fp8(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            flat_page_table.data_ptr(), flat_kv_lens.data_ptr(), R, Hq, Hkv, D, topk, P, o.data_ptr(),
            None if lse is None else lse.data_ptr(), ws, nbytes, stream))
    _lib.check("msa_paged_sparse_decode_fp8", rc)
    return o, lse


def prefill_bucket(block_ids, nblk: int, workspace: Workspace | None = None):
    """Invert selections into per-(group, block) lists (``msa_prefill_bucket``).

    Returns (offsets [Hkv, nblk+1] int32, entries [T*Hkv*topk] int32; only the first
    sum over groups of offsets[g, nblk] entries are meaningful).
    """
    _need(block_ids, "block_ids", torch.int32, 3)
    T, Hkv, topk = block_ids.shape
    dev = block_ids.device
    offsets = torch.empty((Hkv, nblk + 1), dtype=torch.int32, device=dev)
    entries = torch.empty((max(T * Hkv * topk, 1),), dtype=torch.int32, device=dev)
    lib = load()
    nbytes = lib.msa_prefill_bucket_workspace_size(T, Hkv, topk, nblk)
    buf = _ws(workspace, dev).get("bucket", nbytes, dev)
    rc = lib.msa_prefill_bucket(_ptr(block_ids), T, Hkv, topk, nblk, _ptr(offsets), _ptr(entries),
                                _ptr(buf), buf.numel(), _stream(dev))
    _lib.check("msa_prefill_bucket", rc)
    return offsets, entries


def lse_merge(o_parts, lse_parts, with_lse: bool = True):
    """Merge partials o_parts [U, S, G, D] (bf16 or fp32) with lse_parts [U, S, G] fp32."""
    if o_parts.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("lse_merge: o_parts must be bf16 or fp32")
    _need(o_parts, "o_parts", o_parts.dtype, 4)
    _need(lse_parts, "lse_parts", torch.float32, 3)
    U, S, G, D = o_parts.shape
    if lse_parts.shape != (U, S, G):
        raise ValueError("lse_merge: lse_parts shape")
    dev = o_parts.device
    o = torch.empty((U, G, D), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((U, G), dtype=torch.float32, device=dev) if with_lse else None
    rc = load().msa_lse_merge(_ptr(o_parts), 1 if o_parts.dtype == torch.bfloat16 else 0,
                              _ptr(lse_parts), U, S, G, D, _ptr(o), _ptr(lse), _stream(dev))
    _lib.check("msa_lse_merge", rc)
    return o, lse


def device_error() -> int:
    """Synchronise and return (then clear) the kernels' device error word (0 = none)."""
    w = ctypes.c_uint32(0)
    rc = load().msa_device_error(ctypes.byref(w))
    if rc not in (0, -6):
        _lib.check("msa_device_error", rc)
    return int(w.value)
