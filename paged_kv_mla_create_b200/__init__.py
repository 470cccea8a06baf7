"""Paged MLA decode for B200 (sm_100a): page table, split-KV planner and attention.

A thin ctypes binding over the in-tree C-ABI library ``libmla_b200.so`` (declared in
``include/mla_b200.h``).  Every function here only marshals torch tensors into device
pointers and the current CUDA stream; all arithmetic runs in the library's kernels.
There is no CPU fallback: without the library, or without a CUDA device, the calls
raise.

The three entry points follow the calls of the SGLang FlashMLA attention backend page
(flashmla_backend.py):

* ``build_block_table``   — ``create_flashmla_kv_indices_triton`` in
  ``init_forward_metadata`` (block_kv_indices [bs, cdiv(max L, 64)], -1 padded);
* ``get_mla_metadata``    — ``get_mla_metadata(seq_lens, num_heads_per_head_k,
  num_heads_k, is_fp8_kvcache)`` returning (tile_scheduler_metadata, num_splits);
* ``mla_decode_paged``    — ``flash_mla_with_kvcache(q, k_cache, block_table,
  cache_seqlens, head_dim_v, tile_scheduler_metadata, num_splits, softmax_scale,
  causal, descale_q, descale_k)`` returning (o, lse); also exported under that name.

For requests that bring different numbers of new tokens: ``build_chunk_metadata`` (page table, lengths,
positions, pool slots and plan from the requests' lengths), ``set_kv_buffer``, ``mla_chunk_paged``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

from . import build as _build

__all__ = [
    "build_block_table", "get_mla_metadata", "build_decode_metadata", "mla_decode_paged",
    "flash_mla_with_kvcache", "set_kv_buffer", "build_chunk_metadata", "mla_chunk_paged",
    "num_chunk_parts", "chunk_workspace_bytes",
    "num_sm_parts", "workspace_bytes", "read_device_error", "library", "MlaError",
]

PAGE_SIZE = 64
_STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_CUDA",
           4: "MLA_ERR_DEVICE_CHECK", 5: "MLA_ERR_WORKSPACE"}
DTYPE_BF16, DTYPE_FP8_E4M3, DTYPE_INT32, DTYPE_INT64, DTYPE_FP8_E5M2 = 0, 1, 2, 3, 4
_CACHE_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float8_e4m3fn: DTYPE_FP8_E4M3,
                 torch.float8_e5m2: DTYPE_FP8_E5M2}

_lib = None


class MlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(status, status)}")
        self.status = status


def library() -> ctypes.CDLL:
    """Load (building first when stale) the CUDA library; raises when it cannot."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if _build.is_stale():
        path = _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library missing: {path}")
    lib = ctypes.CDLL(path)
    P, I32, I64, F, SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                          ctypes.c_size_t)
    lib.mla_status_string.argtypes = [I32]
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_abi_version.argtypes = []
    lib.mla_abi_version.restype = I32
    lib.mla_build_block_table.argtypes = [P, I64, I64, P, I32, P, I32, I32, I32, P, I64, I32, I32,
                                          I32, P]
    lib.mla_build_block_table.restype = I32
    lib.mla_num_sm_parts.argtypes = [I32, I32, I32]
    lib.mla_num_sm_parts.restype = I32
    lib.mla_get_mla_metadata.argtypes = [P, I32, I32, I32, I32, I32, P, P, P]
    lib.mla_get_mla_metadata.restype = I32
    lib.mla_build_decode_metadata.argtypes = [P, I64, I64, P, I32, P, I32, I32, I32, P, I64, I32,
                                              I32, I32, I32, I32, I32, I32, P, P, P, P]
    lib.mla_build_decode_metadata.restype = I32
    lib.mla_decode_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.mla_decode_workspace_bytes.restype = SZ
    lib.mla_decode_paged.argtypes = [P, I32, I32, I32, I32, I32, I32, P, I32, I64, I32, P, I64,
                                     I32, P, P, I32, P, F, I32, P, P, P, P, P, SZ, P]
    lib.mla_decode_paged.restype = I32
    lib.mla_set_kv_buffer.argtypes = [P, I32, I64, P, I32, I32, P, I64, P, P]
    lib.mla_set_kv_buffer.restype = I32
    lib.mla_merge_state.argtypes = [P, P, P, P, I64, I32, P, P, P]
    lib.mla_merge_state.restype = I32
    lib.mla_extend_workspace_bytes.argtypes = [I32, I32, I32, I32, I32]
    lib.mla_extend_workspace_bytes.restype = ctypes.c_size_t
    lib.mla_extend_paged_prefix.argtypes = [P, I32, I32, I32, P, P, I32, I64, P, I64, I64, P, I32, P, I32,
                                            ctypes.c_float, P, I32, P, P, P, ctypes.c_size_t, P]
    lib.mla_extend_paged_prefix.restype = I32
    lib.mla_build_chunk_metadata.argtypes = [P, I64, I64, P, I32, P, P, I32, I32, I32, P, I64, I32, I32, I32, P, I64, I32,
                                             I32, I32, I32, P, P, P, P, P, P, P]
    lib.mla_build_chunk_metadata.restype = I32
    lib.mla_build_chunk_metadata_view.argtypes = [P, I64, I64, I64, P, I32, P, P, I32, I32, I32, P, I64, I32, I32, I32, P, I64,
                                                  I32, I32, I32, I32, P, P, P, P, P, P, P]
    lib.mla_build_chunk_metadata_view.restype = I32
    lib.mla_num_chunk_parts.argtypes = [I32]
    lib.mla_num_chunk_parts.restype = I32
    lib.mla_chunk_workspace_bytes.argtypes = [I32]
    lib.mla_chunk_workspace_bytes.restype = SZ
    lib.mla_chunk_paged.argtypes = [P, I32, I32, I32, I32, I32, P, I32, I64, I32, P, I64, I32, P, P, I32, P, I32, F, I32,
                                    P, P, P, P, P, SZ, P]
    lib.mla_chunk_paged.restype = I32
    lib.mla_set_test_hooks.argtypes = [ctypes.c_uint64, I32, I32]
    lib.mla_set_test_hooks.restype = I32
    lib.mla_read_device_error.argtypes = [ctypes.POINTER(I32), P]
    lib.mla_read_device_error.restype = I32
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        raise MlaError(status, what)


# The address of a device's current stream without a Stream object (a private name, as torch's own
# generated code uses it; without it the public call does the same a few microseconds slower).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(device) -> ctypes.c_void_p:
    """The device's current stream (device: a torch.device, its name or an index)."""
    if isinstance(device, str):
        device = torch.device(device)
    index = device if isinstance(device, int) else device.index
    return ctypes.c_void_p(_raw_stream(torch.cuda.current_device() if index is None else index))


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _addr(t: Optional[torch.Tensor]) -> Optional[int]:
    """A tensor's address as the plain number that ctypes takes for a pointer (cheaper than an object)."""
    return t.data_ptr() if t is not None else None


@functools.lru_cache(maxsize=None)
def _device_parts(index: int) -> int:
    """num_chunk_parts of a device."""
    return num_chunk_parts(sm_count(index))


def _on(device: torch.device):
    """A context with `device` current, or none where it is already (the switch costs microseconds)."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _same_device(device: torch.device, *tensors) -> None:
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("all tensors must be on the same CUDA device")


def _require_cuda(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("paged_kv_mla_create_b200 runs on CUDA tensors only")


def _index_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.int32:
        return DTYPE_INT32
    if t.dtype == torch.int64:
        return DTYPE_INT64
    raise ValueError(f"index tensors must be int32 or int64, got {t.dtype}")


def sm_count(device=None) -> int:
    return torch.cuda.get_device_properties(torch.cuda.current_device() if device is None else device).multi_processor_count


def num_sm_parts(num_heads_per_head_k: int, num_heads_k: int = 1,
                 sm_count_: Optional[int] = None) -> int:
    """Rows of tile_scheduler_metadata for q_len * h_q = num_heads_per_head_k."""
    n = library().mla_num_sm_parts(sm_count_ if sm_count_ is not None else sm_count(),
                                   num_heads_per_head_k, num_heads_k)
    if n < 1:
        raise ValueError("invalid arguments to num_sm_parts")
    return n


def workspace_bytes(bs: int, q_len: int, h_q: int, parts: int) -> int:
    """Bytes of the attention workspace; allocate it zero-filled (torch.zeros) once, then
    reuse it: every completed call leaves its leading arrival words zero."""
    return int(library().mla_decode_workspace_bytes(bs, q_len, h_q, parts))


def _map_pages(req_to_token: torch.Tensor, max_pages: int) -> int:
    """Pages a row of req_to_token has slots for, at most max_pages.  The library takes the row pitch for the
    width; where the map is part of a wider matrix, the columns that are not its own are never asked for."""
    if req_to_token.shape[1] >= req_to_token.stride(0):
        return max_pages
    return min(max_pages, -(-req_to_token.shape[1] // PAGE_SIZE))


def build_block_table(req_to_token: torch.Tensor, req_pool_indices: torch.Tensor,
                      seq_lens: torch.Tensor, max_seqlen_pad: int, seq_len_add: int = 0,
                      out: Optional[torch.Tensor] = None, fill_tail: bool = True) -> torch.Tensor:
    """int32 [bs, max_seqlen_pad] page table: entry (b, p) is the page holding position 64p
    of request b (L_b = seq_lens[b] + seq_len_add); other entries are -1 when fill_tail."""
    _require_cuda(req_to_token, req_pool_indices, seq_lens, out)
    if req_to_token.dtype != torch.int32 or req_to_token.dim() != 2 or req_to_token.stride(1) != 1:
        raise ValueError("req_to_token must be a row-major int32 matrix")
    bs = int(req_pool_indices.shape[0])
    if out is None:
        out = torch.empty((bs, max_seqlen_pad), dtype=torch.int32, device=req_to_token.device)
    if out.dtype != torch.int32 or out.dim() != 2 or out.stride(1) != 1:
        raise ValueError("out must be a row-major int32 matrix")
    rpi = req_pool_indices.contiguous()
    sl = seq_lens.contiguous()
    pages = _map_pages(req_to_token, int(max_seqlen_pad))
    if fill_tail and pages < max_seqlen_pad:
        out[:bs, pages:max_seqlen_pad] = -1
    _check(library().mla_build_block_table(
        _ptr(req_to_token), req_to_token.shape[0], req_to_token.stride(0), _ptr(rpi),
        _index_dtype(rpi), _ptr(sl), _index_dtype(sl), int(seq_len_add), bs, _ptr(out),
        out.stride(0), pages, PAGE_SIZE, int(bool(fill_tail)),
        _stream(req_to_token.device)), "mla_build_block_table")
    return out


def get_mla_metadata(cache_seqlens: torch.Tensor, num_heads_per_head_k: int,
                     num_heads_k: int = 1, is_fp8_kvcache: bool = False,
                     num_parts: Optional[int] = None,
                     out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """(tile_scheduler_metadata int32 [num_sm_parts, 8], num_splits int32 [bs + 1]).

    The part count follows from the device's SM count; ``num_parts`` plans for that many
    parts instead (the SM count of a device with 2 SMs per part and query tile)."""
    _require_cuda(cache_seqlens)
    if cache_seqlens.dtype != torch.int32:
        raise ValueError("cache_seqlens must be int32 (the backend casts with .to(torch.int32))")
    if num_heads_per_head_k <= 0 or num_heads_k <= 0:
        raise ValueError("num_heads_per_head_k and num_heads_k must be positive")
    sl = cache_seqlens.contiguous()
    bs = int(sl.shape[0])
    dev = sl.device
    if num_parts is not None:
        m_tiles = -(-num_heads_per_head_k // 128)
        sms = 2 * m_tiles * num_heads_k * int(num_parts)
    else:
        sms = sm_count(dev)
    parts = num_sm_parts(num_heads_per_head_k, num_heads_k, sms)
    if out is None:
        md = torch.empty((parts, 8), dtype=torch.int32, device=dev)
        ns = torch.empty((bs + 1,), dtype=torch.int32, device=dev)
    else:
        md, ns = out
        if md.shape[0] != parts or ns.numel() != bs + 1:
            raise ValueError("out tensors do not match the plan's shapes")
    _check(library().mla_get_mla_metadata(_ptr(sl), bs, int(num_heads_per_head_k), int(num_heads_k),
                                          int(bool(is_fp8_kvcache)), sms, _ptr(md), _ptr(ns),
                                          _stream(dev)),
           "mla_get_mla_metadata")
    return md, ns


def build_decode_metadata(req_to_token: torch.Tensor, req_pool_indices: torch.Tensor,
                          seq_lens: torch.Tensor, max_seqlen_pad: int, num_heads_per_head_k: int,
                          num_heads_k: int = 1, is_fp8_kvcache: bool = False, seq_len_add: int = 0,
                          num_parts: Optional[int] = None, fill_tail: bool = True,
                          out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]] = None):
    """The per-batch metadata in one launch: (block_table int32 [bs, max_seqlen_pad],
    cache_seqlens int32 [bs] = seq_lens + seq_len_add, tile_scheduler_metadata int32
    [num_sm_parts, 8], num_splits int32 [bs + 1]) -- what build_block_table, the int32 cast
    of the lengths and get_mla_metadata give."""
    _require_cuda(req_to_token, req_pool_indices, seq_lens)
    if req_to_token.dtype != torch.int32 or req_to_token.dim() != 2 or req_to_token.stride(1) != 1:
        raise ValueError("req_to_token must be a row-major int32 matrix")
    if num_heads_per_head_k <= 0 or num_heads_k <= 0:
        raise ValueError("num_heads_per_head_k and num_heads_k must be positive")
    dev = req_to_token.device
    bs = int(req_pool_indices.shape[0])
    if num_parts is not None:
        sms = 2 * (-(-num_heads_per_head_k // 128)) * num_heads_k * int(num_parts)
    else:
        sms = sm_count(dev)
    parts = num_sm_parts(num_heads_per_head_k, num_heads_k, sms)
    if out is None:
        bt = torch.empty((bs, max_seqlen_pad), dtype=torch.int32, device=dev)
        cl = torch.empty((bs,), dtype=torch.int32, device=dev)
        md = torch.empty((parts, 8), dtype=torch.int32, device=dev)
        ns = torch.empty((bs + 1,), dtype=torch.int32, device=dev)
    else:
        bt, cl, md, ns = out
    if bt.dtype != torch.int32 or bt.dim() != 2 or bt.stride(1) != 1:
        raise ValueError("block_table must be a row-major int32 matrix")
    if md.shape[0] != parts or ns.numel() != bs + 1 or (cl is not None and cl.numel() != bs):
        raise ValueError("out tensors do not match the metadata's shapes")
    rpi = req_pool_indices.contiguous()
    sl = seq_lens.contiguous()
    pages = _map_pages(req_to_token, int(max_seqlen_pad))
    if fill_tail and pages < max_seqlen_pad:
        bt[:bs, pages:max_seqlen_pad] = -1
    _check(library().mla_build_decode_metadata(
        _ptr(req_to_token), req_to_token.shape[0], req_to_token.stride(0), _ptr(rpi),
        _index_dtype(rpi), _ptr(sl), _index_dtype(sl), int(seq_len_add), bs, _ptr(bt), bt.stride(0),
        pages, PAGE_SIZE, int(bool(fill_tail)), int(num_heads_per_head_k),
        int(num_heads_k), int(bool(is_fp8_kvcache)), sms, _ptr(cl), _ptr(md), _ptr(ns),
        _stream(dev)), "mla_build_decode_metadata")
    return bt, cl, md, ns


def mla_decode_paged(q: torch.Tensor, k_cache: torch.Tensor, block_table: torch.Tensor,
                     cache_seqlens: torch.Tensor, head_dim_v: int,
                     tile_scheduler_metadata: torch.Tensor, num_splits: torch.Tensor,
                     softmax_scale: float, causal: bool = True,
                     descale_q: Optional[torch.Tensor] = None,
                     descale_k: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Paged MLA attention.  q bf16 [bs, q_len, h_q, 576], or float8_e4m3fn codes with an
    float8_e4m3fn cache (the backend's fp8 branch: q quantised with the cache's scale, that
    scale passed as descale_q and descale_k); k_cache bf16 or float8_e4m3fn with 576-wide
    token rows grouped in 64-token pages ([pages, 64, 576], [pages, 64, 1, 576] or
    [slots, 576]).  Returns (o bf16 [bs, q_len, h_q, 512], lse fp32 [bs, q_len, h_q])."""
    _require_cuda(q, k_cache, block_table, cache_seqlens, tile_scheduler_metadata, num_splits,
                  descale_q, descale_k, out, lse, workspace)
    if q.dim() != 4 or q.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 or float8_e4m3fn [bs, q_len, h_q, head_dim] tensor")
    bs, q_len, h_q, head_dim = (int(x) for x in q.shape)
    if not k_cache.is_contiguous() or k_cache.shape[-1] != head_dim:
        raise ValueError("k_cache must be contiguous with head_dim-wide rows")
    if k_cache.numel() % (PAGE_SIZE * head_dim):
        raise ValueError("k_cache must hold whole 64-token pages")
    num_pages = k_cache.numel() // (PAGE_SIZE * head_dim)
    if k_cache.dtype not in _CACHE_DTYPES:
        raise ValueError(f"unsupported k_cache dtype {k_cache.dtype}")
    kv_dtype = _CACHE_DTYPES[k_cache.dtype]
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be a row-major int32 [bs, max_pages] matrix")
    if cache_seqlens.dtype != torch.int32:
        raise ValueError("cache_seqlens must be int32")
    for name, d in (("descale_q", descale_q), ("descale_k", descale_k)):
        if d is not None and (d.dtype != torch.float32 or d.numel() < 1):
            raise ValueError(f"{name} must be a float32 tensor of one element")
    dev = q.device
    parts = int(tile_scheduler_metadata.shape[0])
    if out is None:
        out = torch.empty((bs, q_len, h_q, head_dim_v), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((bs, q_len, h_q), dtype=torch.float32, device=dev)
    need = workspace_bytes(bs, q_len, h_q, parts) if bs else 0
    if workspace is None and need:
        # zero-filled: the leading arrival words must be zero at a workspace's first use
        workspace = torch.zeros((need,), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    sl = cache_seqlens.contiguous()
    q_dtype = DTYPE_FP8_E4M3 if q.dtype == torch.float8_e4m3fn else DTYPE_BF16
    _check(library().mla_decode_paged(
        _ptr(q), q_dtype, bs, q_len, h_q, head_dim, int(head_dim_v), _ptr(k_cache), kv_dtype,
        num_pages, PAGE_SIZE, _ptr(block_table), block_table.stride(0), int(block_table.shape[1]),
        _ptr(sl), _ptr(tile_scheduler_metadata), parts, _ptr(num_splits), float(softmax_scale),
        int(bool(causal)), _ptr(descale_q), _ptr(descale_k), _ptr(out), _ptr(lse),
        _ptr(workspace), ws_bytes, _stream(dev)), "mla_decode_paged")
    return out, lse


flash_mla_with_kvcache = mla_decode_paged


def set_kv_buffer(k_cache: torch.Tensor, cache_loc: torch.Tensor, k: torch.Tensor,
                  k_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """token_to_kv_pool.set_kv_buffer for the MLA latent pool: row cache_loc[i] of k_cache
    ([slots, 576] or any view with 576-wide rows; bf16, float8_e4m3fn or float8_e5m2) receives
    k[i] (bf16 [n, 576], the latent row whose first 512 columns are the value), an fp8 pool
    storing k / k_scale rounded to its format.  In place; returns k_cache."""
    _require_cuda(k_cache, cache_loc, k, k_scale)
    if k_cache.dtype not in _CACHE_DTYPES or not k_cache.is_contiguous() or k_cache.shape[-1] != 576:
        raise ValueError("k_cache must be a contiguous bf16 / float8 pool with 576-wide rows")
    if k.dtype != torch.bfloat16 or k.dim() != 2 or k.shape[1] != 576 or k.stride(1) != 1:
        raise ValueError("k must be a bf16 [n, 576] matrix with unit column stride")
    if k_scale is not None and (k_scale.dtype != torch.float32 or k_scale.numel() < 1):
        raise ValueError("k_scale must be a float32 tensor of one element")
    loc = cache_loc.contiguous()
    n = int(k.shape[0])
    if loc.numel() != n:
        raise ValueError("one cache_loc entry per token")
    _check(library().mla_set_kv_buffer(_ptr(k_cache), _CACHE_DTYPES[k_cache.dtype], k_cache.numel() // 576,
                                       _ptr(loc), _index_dtype(loc), n, _ptr(k), k.stride(0), _ptr(k_scale),
                                       _stream(k_cache.device)), "mla_set_kv_buffer")
    return k_cache


def merge_state(o_a: torch.Tensor, lse_a: torch.Tensor, o_b: torch.Tensor, lse_b: torch.Tensor,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """merge_state(o1, s1, o2, s2) of two partial attention results of the same rows: bf16
    o [..., 512] and fp32 natural-log lse [...] (-inf: no key).  Returns (o, lse)."""
    _require_cuda(o_a, lse_a, o_b, lse_b, out, lse)
    for o_, l_ in ((o_a, lse_a), (o_b, lse_b)):
        if o_.dtype != torch.bfloat16 or not o_.is_contiguous() or o_.shape[-1] != 512:
            raise ValueError("o must be a contiguous bf16 [..., 512] tensor")
        if l_.dtype != torch.float32 or not l_.is_contiguous() or l_.numel() * 512 != o_.numel():
            raise ValueError("lse must be a contiguous float32 tensor of one value per row")
    if o_a.shape != o_b.shape:
        raise ValueError("the two parts must have the same shape")
    rows = lse_a.numel()
    if out is None:
        out = torch.empty_like(o_a)
    if lse is None:
        lse = torch.empty_like(lse_a)
    _check(library().mla_merge_state(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), rows, 512, _ptr(out), _ptr(lse),
                                     _stream(o_a.device)), "mla_merge_state")
    return out, lse


def extend_workspace_bytes(bs: int, e: int, h_q: int, max_prefix_pages: int, sm_count_: Optional[int] = None) -> int:
    """Bytes of the extend workspace; allocate it zero-filled once and reuse it."""
    return int(library().mla_extend_workspace_bytes(bs, e, h_q, max_prefix_pages,
                                                    sm_count_ if sm_count_ is not None else sm_count()))


def extend_paged_prefix(q: torch.Tensor, k_new: torch.Tensor, k_cache: torch.Tensor, req_to_token: torch.Tensor,
                        req_pool_indices: torch.Tensor, prefix_lens: torch.Tensor, max_prefix_pages: int,
                        softmax_scale: float, descale_k: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """Extend with a cached prefix: q bf16 [bs, e, h_q, 576] of the e new tokens of every request
    attends the new tokens' latent rows k_new (bf16 [bs, e, 576]) causally and the request's
    prefix_lens[b] cached rows of k_cache (through req_to_token) in full; the two partial results
    are merged by merge_state.  Returns (o bf16 [bs, e, h_q, 512], lse fp32 [bs, e, h_q])."""
    _require_cuda(q, k_new, k_cache, req_to_token, req_pool_indices, prefix_lens, descale_k, out, lse, workspace)
    if q.dim() != 4 or q.dtype != torch.bfloat16 or not q.is_contiguous() or q.shape[-1] != 576:
        raise ValueError("q must be a contiguous bf16 [bs, e, h_q, 576] tensor")
    bs, e, h_q, _ = (int(x) for x in q.shape)
    if k_new.dtype != torch.bfloat16 or not k_new.is_contiguous() or tuple(k_new.shape) != (bs, e, 576):
        raise ValueError("k_new must be a contiguous bf16 [bs, e, 576] tensor")
    if k_cache.dtype not in _CACHE_DTYPES or not k_cache.is_contiguous() or k_cache.shape[-1] != 576:
        raise ValueError("k_cache must be a contiguous bf16 / float8 pool with 576-wide rows")
    if k_cache.numel() % (PAGE_SIZE * 576):
        raise ValueError("k_cache must hold whole 64-token pages")
    if req_to_token.dtype != torch.int32 or req_to_token.dim() != 2 or req_to_token.stride(1) != 1:
        raise ValueError("req_to_token must be a row-major int32 matrix")
    pl = prefix_lens.to(torch.int32).contiguous()
    rpi = req_pool_indices.contiguous()
    dev = q.device
    if out is None:
        out = torch.empty((bs, e, h_q, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((bs, e, h_q), dtype=torch.float32, device=dev)
    pages = _map_pages(req_to_token, int(max_prefix_pages))
    need = extend_workspace_bytes(bs, e, h_q, pages) if bs else 0
    if workspace is None and need:
        workspace = torch.zeros((need,), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(library().mla_extend_paged_prefix(
        _ptr(q), bs, e, h_q, _ptr(k_new), _ptr(k_cache), _CACHE_DTYPES[k_cache.dtype],
        k_cache.numel() // (PAGE_SIZE * 576), _ptr(req_to_token), int(req_to_token.shape[0]),
        req_to_token.stride(0), _ptr(rpi), _index_dtype(rpi), _ptr(pl), pages,
        float(softmax_scale), _ptr(descale_k), sm_count(dev), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
        _stream(dev)), "mla_extend_paged_prefix")
    return out, lse


def num_chunk_parts(sm_count_: Optional[int] = None) -> int:
    """Rows of a chunk plan (build_chunk_metadata): one per pair of SMs."""
    n = library().mla_num_chunk_parts(sm_count_ if sm_count_ is not None else sm_count())
    if n < 1:
        raise ValueError("invalid argument to num_chunk_parts")
    return n


def chunk_workspace_bytes(parts: int) -> int:
    """Bytes of the ragged attention's workspace for a plan of `parts` rows (no initialisation needed)."""
    n = int(library().mla_chunk_workspace_bytes(int(parts)))
    if n == 0:
        raise ValueError("a chunk plan has between 1 and 1024 parts")
    return n


def _int32_vector(t: torch.Tensor, name: str, least: int) -> None:
    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < least:
        raise ValueError(f"{name} must be a contiguous int32 tensor of at least {least} elements")


def build_chunk_metadata(req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, prefix_lens: torch.Tensor,
                         chunk_lens: torch.Tensor, num_tokens: int, max_seqlen_pad: int, num_heads: int,
                         free_pages: Optional[torch.Tensor] = None, causal: bool = True, pad_slot: int = -1,
                         fill_tail: bool = True, num_parts: Optional[int] = None,
                         out: Optional[Tuple[torch.Tensor, ...]] = None):
    """Metadata of a ragged batch in one launch: request b has prefix_lens[b] cached tokens and
    brings chunk_lens[b] new ones, their rows one request after another in num_tokens rows.
    Returns (block_table int32 [bs, max_seqlen_pad], cache_seqlens int32 [bs], cu_seqlens int32
    [bs + 1], positions int32 [num_tokens], cache_loc int32 [num_tokens], chunk_plan int32 [parts, 8],
    pages_taken int32 [1], or None without free_pages).

    Without free_pages the new tokens' slots are read from req_to_token; with them new pages are
    taken from the list, in request order, and the new slots entered into req_to_token (the
    requests' rows must differ then).  Rows behind the last request get position 0 and slot
    pad_slot when fill_tail (-1: not a slot; set_kv_buffer skips and reports it), else nothing.

    out: the tensors to write, in the order of the result; all but the plan, whose rows are the parts',
    may be larger."""
    if not req_to_token.is_cuda:
        raise ValueError("paged_kv_mla_create_b200 runs on CUDA tensors only")
    dev = req_to_token.device
    _same_device(dev, req_pool_indices, prefix_lens, chunk_lens, free_pages, *(out or ()))
    if req_to_token.dtype != torch.int32 or req_to_token.dim() != 2 or req_to_token.stride(1) != 1:
        raise ValueError("req_to_token must be a row-major int32 matrix")
    if num_tokens < 0 or max_seqlen_pad < 0 or num_heads <= 0:
        raise ValueError("num_tokens and max_seqlen_pad must not be negative, num_heads must be positive")
    if max(num_tokens, max_seqlen_pad, num_heads, abs(pad_slot), num_parts or 0) > 0x7FFFFFFF:
        raise ValueError("num_tokens, max_seqlen_pad, num_heads, pad_slot and num_parts must fit into 32 bits")
    bs = req_pool_indices.shape[0]
    if not (req_pool_indices.shape == prefix_lens.shape == chunk_lens.shape == (bs,)):
        raise ValueError("req_pool_indices, prefix_lens and chunk_lens must be vectors of one entry per request")
    if prefix_lens.dtype != chunk_lens.dtype:
        raise ValueError("prefix_lens and chunk_lens must have the same dtype")
    rpi, pl, cl = req_pool_indices.contiguous(), prefix_lens.contiguous(), chunk_lens.contiguous()
    if free_pages is not None:
        if free_pages.dim() != 1 or free_pages.dtype != rpi.dtype:
            raise ValueError("free_pages must be a vector of req_pool_indices' dtype")
        free_pages = free_pages.contiguous()
    parts = _device_parts(dev.index) if num_parts is None else int(num_parts)
    if out is None:
        # one allocation for all of them, the plan (16-byte aligned) first
        sizes = (8 * max(parts, 0), bs * max_seqlen_pad, bs, bs + 1, num_tokens, num_tokens, 1)
        plan, bt, seqlens, cu, positions, loc, taken = torch.empty(
            sum(sizes), dtype=torch.int32, device=dev).split_with_sizes(sizes)
        out = (bt.view(bs, max_seqlen_pad), seqlens, cu, positions, loc, plan.view(max(parts, 0), 8),
               taken if free_pages is not None else None)
    else:
        bt, seqlens, cu, positions, loc, plan, taken = out
        if bt.dtype != torch.int32 or bt.dim() != 2 or bt.stride(1) != 1 or bt.shape[0] < bs or bt.shape[1] < max_seqlen_pad:
            raise ValueError("block_table must be a row-major int32 [bs, max_seqlen_pad] matrix")
        _int32_vector(seqlens, "cache_seqlens", bs)
        _int32_vector(cu, "cu_seqlens", bs + 1)
        _int32_vector(positions, "positions", num_tokens)
        _int32_vector(loc, "cache_loc", num_tokens)
        _int32_vector(plan, "chunk_plan", 8 * parts)
        if plan.numel() != 8 * parts:   # the attention would run rows behind the last as parts
            raise ValueError(f"chunk_plan must have a row for each of the {parts} parts and no other")
        if taken is not None:
            _int32_vector(taken, "pages_taken", 1)
    bt, taken = out[0], out[6]
    map_rows, map_cols = req_to_token.shape
    # a free list without entries is still a list (its data pointer may be null)
    free_ptr = None if free_pages is None else free_pages.data_ptr() or rpi.data_ptr()
    with _on(dev):
        _check(library().mla_build_chunk_metadata_view(
            _addr(req_to_token), map_rows, req_to_token.stride(0), map_cols, _addr(rpi), _index_dtype(rpi), _addr(pl),
            _addr(cl), _index_dtype(pl), bs, int(num_tokens), free_ptr,
            free_pages.shape[0] if free_pages is not None else 0, int(num_heads), int(bool(causal)), parts, _addr(bt),
            bt.stride(0), int(max_seqlen_pad), PAGE_SIZE, int(bool(fill_tail)), int(pad_slot), _addr(seqlens), _addr(cu),
            _addr(positions), _addr(loc), _addr(plan), _addr(taken), _stream(dev)), "mla_build_chunk_metadata")
    return out


def mla_chunk_paged(q: torch.Tensor, k_cache: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
                    cu_seqlens: torch.Tensor, head_dim_v: int, chunk_plan: torch.Tensor, softmax_scale: float,
                    causal: bool = True, descale_q: Optional[torch.Tensor] = None,
                    descale_k: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Paged MLA attention of ragged chunks: rows [cu_seqlens[b], cu_seqlens[b + 1]) of q (bf16
    [num_tokens, h_q, 576]) are request b's new tokens, the last of its cache_seqlens[b] cached rows;
    each sees the rows up to its own (causal) or all of them.  Lengths, offsets and plan as
    build_chunk_metadata gives them for h_q heads and the same causal; k_cache bf16, float8_e4m3fn or
    float8_e5m2.  Returns (o bf16 [num_tokens, h_q, 512], lse fp32 [num_tokens, h_q]); rows of no
    request keep what out / lse held."""
    if not q.is_cuda:
        raise ValueError("paged_kv_mla_create_b200 runs on CUDA tensors only")
    dev = q.device
    _same_device(dev, k_cache, block_table, cache_seqlens, cu_seqlens, chunk_plan, descale_q, descale_k, out, lse, workspace)
    if q.dim() != 3 or q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 [num_tokens, h_q, head_dim] tensor")
    num_tokens, h_q, head_dim = (int(x) for x in q.shape)
    if not k_cache.is_contiguous() or k_cache.shape[-1] != head_dim:
        raise ValueError("k_cache must be contiguous with head_dim-wide rows")
    if k_cache.numel() % (PAGE_SIZE * head_dim):
        raise ValueError("k_cache must hold whole 64-token pages")
    if k_cache.dtype not in _CACHE_DTYPES:
        raise ValueError(f"unsupported k_cache dtype {k_cache.dtype}")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be a row-major int32 [bs, max_pages] matrix")
    bs = int(block_table.shape[0])
    _int32_vector(cache_seqlens, "cache_seqlens", bs)
    _int32_vector(cu_seqlens, "cu_seqlens", bs + 1)
    if chunk_plan.dtype != torch.int32 or chunk_plan.dim() != 2 or chunk_plan.shape[1] != 8 or not chunk_plan.is_contiguous():
        raise ValueError("chunk_plan must be a contiguous int32 [parts, 8] matrix")
    for name, d in (("descale_q", descale_q), ("descale_k", descale_k)):
        if d is not None and (d.dtype != torch.float32 or d.numel() < 1):
            raise ValueError(f"{name} must be a float32 tensor of one element")
    if out is not None and (out.dtype != torch.bfloat16 or not out.is_contiguous()
                            or tuple(out.shape) != (num_tokens, h_q, head_dim_v)):
        raise ValueError("out must be a contiguous bf16 [num_tokens, h_q, head_dim_v] tensor")
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (num_tokens, h_q)):
        raise ValueError("lse must be a contiguous float32 [num_tokens, h_q] tensor")
    if workspace is not None and not workspace.is_contiguous():   # (an expanded one has fewer bytes than elements)
        raise ValueError("workspace must be contiguous")
    parts = int(chunk_plan.shape[0])
    with _on(dev):
        if out is None:
            out = torch.empty((num_tokens, h_q, head_dim_v), dtype=torch.bfloat16, device=dev)
        if lse is None:
            lse = torch.empty((num_tokens, h_q), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty((chunk_workspace_bytes(parts),), dtype=torch.uint8, device=dev)
        _check(library().mla_chunk_paged(
            _addr(q), DTYPE_BF16, num_tokens, h_q, head_dim, int(head_dim_v), _addr(k_cache), _CACHE_DTYPES[k_cache.dtype],
            k_cache.numel() // (PAGE_SIZE * head_dim), PAGE_SIZE, _addr(block_table), block_table.stride(0),
            int(block_table.shape[1]), _addr(cache_seqlens), _addr(cu_seqlens), bs, _addr(chunk_plan), parts,
            float(softmax_scale), int(bool(causal)), _addr(descale_q), _addr(descale_k), _addr(out), _addr(lse),
            _addr(workspace), workspace.numel() * workspace.element_size(), _stream(dev)), "mla_chunk_paged")
    return out, lse


def set_test_hooks(wait_budget_ns: int = 0, withhold_tile: int = -1, no_fold_in: bool = False) -> None:
    """Test-only: the pipeline wait budget (0: the default 2 s), a tile whose page load the
    leader CTAs withhold (-1: none) and whether the last piece of a split request must merge by
    stored partials instead of folding the others in, for every later attention launch in this
    process."""
    _check(library().mla_set_test_hooks(int(wait_budget_ns), int(withhold_tile), int(bool(no_fold_in))),
           "mla_set_test_hooks")


def read_device_error(device=None) -> int:
    """Synchronise the current stream and return (and clear) the sticky device error word."""
    code = ctypes.c_int32(0)
    status = library().mla_read_device_error(ctypes.byref(code),
                                             _stream(torch.cuda.current_device() if device is None else device))
    if status not in (0, 4):
        raise MlaError(status, "mla_read_device_error")
    return int(code.value)
