"""GB300-native decode context parallelism (DCP) hot path: Python binding of libdcp.so.

The three stages of the method run in hand-written sm_103a CUDA kernels behind the C ABI in
``include/dcp.h``; this module only marshals torch tensors (device pointers, sizes, the
current stream) into those calls and turns status codes into exceptions.  There is no CPU
fallback: if ``libdcp.so`` is missing or the GPU is absent the calls raise.

Entry points (same names as the C ABI):
  layer_range              CP layer split ("Serving Macaron-V1 at Scale", 4.1)
  filter_page_indices      source-side page-index filter (6.2, 6.3)
  reshard_pages            CP layer-split -> DCP page reshard, all paths in one launch (2, 6.3, 6.4)
  partial_decode_attn      per-rank paged MLA decode attention -> partial O + LSE (5.2)
  lse_merge                exact LSE merge of the partials (5.2)
  decode_attn_merged       every rank's attention and the merge in one call
  attn_plan                the attention's plan, made once and run per layer (planned=True)
  token_reshard            reshard into the token-interleaved layout ("SGLang's path"); the
                           attention over it: partial_decode_attn / decode_attn_merged(layout="token")
  naive_full_transfer,     the initial design kept as a baseline (6.1): full KV to every DCP rank,
  naive_inplace_shard        then an in-place shard
  pack_pages, unpack_pages one path's pages through a bounded staging buffer (pack_chunks plans it)
  partial_decode_attn_static  the attention without a caller workspace
  prefill_attn             expanded latent attention of packed prompts (192-dim keys, 128-dim values)
  append_kv                new tokens' rows into the pools: rotated, quantised (block scales), paged
  reshard_scales           the block scales of an 8-bit cache's pages along with the reshard
  selftest_wait_timeout    runs the bounded device wait to its limit (failure-path test)
The host-side multi-rank control (bootstrap, size broadcast, consensus prefix, exchange) is in
``decode_context_paged_gb300.control``.
"""
from __future__ import annotations

import ctypes
import os
import re
import sys
from array import array

import torch



def _usable(views) -> bool:
    """Whether the helper was built from this source's kind, for the running torch and Python: it reads
    their objects with the layouts that it was compiled with."""
    return (hasattr(views, "open") and getattr(views, "built_for_torch", "") == re.match(r"\d+(\.\d+)*", torch.__version__)[0]
            and views.built_for_python == sys.hexversion >> 16)


try:  # the questions and calls below in C++ (tensor_views.cpp), where it was built
    from . import _tensor_views as _views
    if not _usable(_views):
        _views = None
except ImportError:
    _views = None

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdcp.so")

DCP_OK = 0
DCP_KV_BF16 = 0
DCP_KV_FP8_E4M3 = 1
DEVERR_OUT_OF_RANGE = 0x1
DEVERR_TIMEOUT = 0x2
DEVERR_PLAN_MISMATCH = 0x4
DEVERR_LAYOUT = 0x8
PAGE = 64
K_DIM = 576
V_DIM = 512

_lib = None
_calls = None  # where the serving calls go: the C++ helper, else the ctypes library


class DcpError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


def _load():
    global _lib, _calls
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(nvcc, sm_103a); there is no fallback path")
        lib = ctypes.CDLL(LIB_PATH)
        i32, i64, f32, vp, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
        lib.dcp_version.restype = i32
        lib.dcp_status_string.argtypes = [i32]
        lib.dcp_status_string.restype = ctypes.c_char_p
        lib.dcp_device_error_status.argtypes = [ctypes.c_int32]
        lib.dcp_device_error_status.restype = i32
        lib.dcp_layer_range.argtypes = [i32, i32, i32, vp, vp]
        lib.dcp_layer_range.restype = i32
        lib.dcp_filter_page_indices.argtypes = [i64, vp, vp, i32, i32, vp, vp, vp, vp]
        lib.dcp_token_reshard.argtypes = [i32, vp, vp, vp, vp, i64, vp, i32, i32, i32, vp, i64, i32, vp, i64, vp, vp]
        lib.dcp_token_reshard.restype = i32
        lib.dcp_naive_full_transfer.argtypes = [i64, vp, i32, i32, i32, vp, i64, i32, vp, vp, vp]
        lib.dcp_naive_full_transfer.restype = i32
        lib.dcp_naive_inplace_shard.argtypes = [i64, vp, i32, i32, i32, vp, vp, i64, vp, vp]
        lib.dcp_naive_inplace_shard.restype = i32
        lib.dcp_pack_pages.argtypes = [i64, vp, i32, i64, i64, i32, vp, i64, vp, sz, vp, vp]
        lib.dcp_pack_pages.restype = i32
        lib.dcp_unpack_pages.argtypes = [i64, vp, i32, i32, i64, i64, i32, vp, sz, vp, i32, i64, vp, vp]
        lib.dcp_unpack_pages.restype = i32
        lib.dcp_filter_page_indices.restype = i32
        lib.dcp_reshard_pages.argtypes = [i32, vp, i64, vp, vp, i32, i32, i32, i32, i32, vp, i64, i32,
                                          vp, i64, i32, i32, vp, vp]
        lib.dcp_reshard_pages.restype = i32
        lib.dcp_append_kv.argtypes = [i32, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i32, i32, f32, i32, vp, i64, vp,
                                      i32, vp, f32, i32, i32, i32, vp, i64, i64, vp, i64, i64, vp, vp]
        lib.dcp_append_kv.restype = i32
        lib.dcp_partial_decode_attn_scaled.argtypes = [i32, i32, i32, vp, vp, vp, i64, vp, i32, f32, i32, vp, i64, vp, i32,
                                                       i32, vp, vp, vp, sz, i32, i32, vp, vp]
        lib.dcp_partial_decode_attn_scaled.restype = i32
        lib.dcp_decode_attn_merged_scaled.argtypes = [i32, i32, i32, vp, vp, vp, i64, vp, i32, i32, f32, f32, i32, vp, i64,
                                                      vp, i32, vp, vp, vp, i32, vp, vp, sz, i32, i32, vp, vp]
        lib.dcp_decode_attn_merged_scaled.restype = i32
        lib.dcp_prefill_attn_workspace_size.argtypes = [i32, i64, i64, i32]
        lib.dcp_prefill_attn_workspace_size.restype = sz
        lib.dcp_prefill_attn.argtypes = [i32, i64, i64, i32, vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, f32,
                                         i32, vp, i32, vp, vp, sz, vp, vp]
        lib.dcp_prefill_attn.restype = i32
        lib.dcp_reshard_scales.argtypes = [i32, vp, i64, vp, vp, i32, i32, i32, vp, i64, i32, vp, i64, vp, vp]
        lib.dcp_reshard_scales.restype = i32
        lib.dcp_partial_decode_attn_workspace_size.argtypes = [i32, i32, i32, i32, i64]
        lib.dcp_partial_decode_attn_workspace_size.restype = sz
        lib.dcp_partial_decode_attn.argtypes = [i32, i32, i32, vp, vp, vp, i64, vp, i32, i32, f32, f32, i32,
                                                vp, i64, i32, vp, vp, vp, sz, vp, vp]
        lib.dcp_partial_decode_attn.restype = i32
        lib.dcp_partial_decode_attn_tokens.argtypes = lib.dcp_partial_decode_attn.argtypes
        lib.dcp_partial_decode_attn_tokens.restype = i32
        lib.dcp_partial_decode_attn_run.argtypes = lib.dcp_partial_decode_attn.argtypes
        lib.dcp_partial_decode_attn_run.restype = i32
        lib.dcp_attn_plan.argtypes = [i32, i32, i32, vp, i64, vp, i32, i32, i64, i32, vp, sz, vp, vp]
        lib.dcp_attn_plan.restype = i32
        lib.dcp_attn_plan_info.argtypes = [i32, i32, i32, i64, i32, i32, vp, sz, vp, vp]
        lib.dcp_attn_plan_info.restype = i32
        lib.dcp_partial_decode_attn_static.argtypes = [i32, i32, i32, vp, vp, vp, i64, vp, i32, i32, f32, f32,
                                                       i32, vp, i64, i32, vp, vp, vp, vp]
        lib.dcp_partial_decode_attn_static.restype = i32
        lib.dcp_decode_attn_merged.argtypes = [i32, i32, i32, vp, vp, vp, i64, vp, i32, i32, f32, f32, i32, vp,
                                               i64, vp, vp, vp, vp, vp, sz, vp, vp]
        lib.dcp_decode_attn_merged.restype = i32
        lib.dcp_decode_attn_merged_run.argtypes = lib.dcp_decode_attn_merged.argtypes
        lib.dcp_decode_attn_merged_run.restype = i32
        lib.dcp_decode_attn_merged_tokens.argtypes = lib.dcp_decode_attn_merged.argtypes
        lib.dcp_decode_attn_merged_tokens.restype = i32
        lib.dcp_lse_merge.argtypes = [i32, i64, i32, vp, vp, vp, vp, vp]
        lib.dcp_lse_merge.restype = i32
        lib.dcp_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp, vp, vp]
        lib.dcp_selftest_wait_timeout.restype = i32
        _calls = _views if _views and _views.open(lib._handle) else lib
        _lib = lib
    return _lib


def _serving():
    """The library for the calls of a serving step."""
    if _calls is None:
        _load()
    return _calls


def library():
    """The loaded ctypes handle of libdcp.so."""
    return _load()


def version() -> int:
    return int(_load().dcp_version())


def status_string(status: int) -> str:
    return _load().dcp_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != DCP_OK:
        raise DcpError(status, what)


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream or None


def _dptr(t: torch.Tensor | None, name: str, dtype=None, device=True) -> int | None:
    if t is None:
        return None
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _kv_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DCP_KV_BF16
    if t.dtype == torch.float8_e4m3fn:
        return DCP_KV_FP8_E4M3
    raise ValueError(f"KV pools must be bfloat16 or float8_e4m3fn, got {t.dtype}")


def _ptr_array(tensors, name) -> ctypes.Array:
    return (ctypes.c_void_p * len(tensors))(*[_dptr(t, f"{name}[{i}]") for i, t in enumerate(tensors)])


def _check_pools(kv_pools) -> tuple[int, int]:
    """Every pool [slots][64][576] of one dtype; returns (slots, dtype code)."""
    if not kv_pools:
        raise ValueError("kv_pools is empty")
    slots = kv_pools[0].shape[0]
    dtype = _kv_code(kv_pools[0])
    for p in kv_pools:
        if p.shape != (slots, PAGE, K_DIM) or p.dtype != kv_pools[0].dtype:
            raise ValueError("every kv pool must be [slots][64][576] of one dtype")
    return slots, dtype


def _check_out(t: torch.Tensor | None, shape: tuple, name: str) -> None:
    """A caller-supplied output must be fp32 of exactly this shape (the kernels write all of it)."""
    if t is not None and (tuple(t.shape) != tuple(shape) or t.dtype != torch.float32):
        raise ValueError(f"{name} must be float32 {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _check_table(requests: int, seq_lens: torch.Tensor | None, req_page_ptr: torch.Tensor) -> None:
    """The attention takes the number of requests from q and reads so many lengths and page offsets."""
    if seq_lens is not None and seq_lens.numel() < requests:
        raise ValueError(f"seq_lens holds {seq_lens.numel()} lengths of {requests} requests")
    if requests > 0 and req_page_ptr.numel() <= requests:
        raise ValueError(f"req_page_ptr holds {req_page_ptr.numel()} offsets, {requests} requests need {requests + 1}")


def _pool_pages(t: torch.Tensor, name: str) -> tuple[int, int]:
    """(layers, pages) of a pool [layers][pages][64][576] (or [pages][64][576] as one layer)."""
    if t.dim() == 4 and tuple(t.shape[2:]) == (PAGE, K_DIM):
        return t.shape[0], t.shape[1]
    if t.dim() == 3 and tuple(t.shape[1:]) == (PAGE, K_DIM):
        return 1, t.shape[0]
    raise ValueError(f"{name} must be [layers][pages][64][576]")


def device_error_status(word: int) -> int:
    return int(_load().dcp_device_error_status(int(word)))


def layer_range(n_layers: int, n_cp: int, r: int) -> tuple[int, int]:
    s, e = ctypes.c_int(0), ctypes.c_int(0)
    _check(_load().dcp_layer_range(n_layers, n_cp, r, ctypes.addressof(s), ctypes.addressof(e)),
           "dcp_layer_range")
    return s.value, e.value


def filter_page_indices(dst_vpages: torch.Tensor, n_dcp: int, d: int,
                        transfer_idx: torch.Tensor | None = None, stream=None):
    """Returns (slots, src or None, count tensor); the first ``count`` entries are valid."""
    n = dst_vpages.numel()
    out_slot = torch.empty(max(n, 1), dtype=torch.int32, device=dst_vpages.device)
    out_src = torch.empty_like(out_slot) if transfer_idx is not None else None
    count = torch.zeros(1, dtype=torch.int64, device=dst_vpages.device)
    _check(_load().dcp_filter_page_indices(n, _dptr(dst_vpages, "dst_vpages", torch.int32),
                                           _dptr(transfer_idx, "transfer_idx", torch.int32), n_dcp, d,
                                           _dptr(out_slot, "out_slot"), _dptr(out_src, "out_src"),
                                           _dptr(count, "count"), _stream(stream)),
           "dcp_filter_page_indices")
    return out_slot, out_src, count


def token_reshard(seq_lens: torch.Tensor, src_page_ptr: torch.Tensor, src_pages: torch.Tensor,
                  tok_page_ptr: torch.Tensor, tok_vpages: torch.Tensor, num_layers: int, src_pools: list,
                  src_pool_pages: int, dst_pools: list, dst_slots_per_rank: int, dev_error: torch.Tensor | None = None,
                  stream=None) -> None:
    """Row gather into the token-interleaved layout (rank d holds tokens d, d + N, ...)."""
    dtype = _kv_code(src_pools[0])
    sp = _ptr_array(src_pools, "src_pools")
    dp = _ptr_array(dst_pools, "dst_pools")
    _check(_load().dcp_token_reshard(seq_lens.numel(), _dptr(seq_lens, "seq_lens", torch.int32),
                                     _dptr(src_page_ptr, "src_page_ptr", torch.int64),
                                     _dptr(src_pages, "src_pages", torch.int32),
                                     _dptr(tok_page_ptr, "tok_page_ptr", torch.int64), tok_vpages.numel(),
                                     _dptr(tok_vpages, "tok_vpages", torch.int32), dtype, num_layers, len(src_pools),
                                     ctypes.addressof(sp), src_pool_pages, len(dst_pools), ctypes.addressof(dp),
                                     dst_slots_per_rank, _dptr(dev_error, "dev_error", torch.int32), _stream(stream)),
           "dcp_token_reshard")


def naive_full_transfer(src_pages: torch.Tensor, num_layers: int, src_pools: list, src_pool_pages: int,
                        recv_bufs: list, dev_error: torch.Tensor | None = None, stream=None) -> None:
    """Baseline: every page of every layer to every DCP rank's receive buffer [L][pages][64][576]."""
    dtype = _kv_code(src_pools[0])
    sp = _ptr_array(src_pools, "src_pools")
    rp = _ptr_array(recv_bufs, "recv_bufs")
    _check(_load().dcp_naive_full_transfer(src_pages.numel(), _dptr(src_pages, "src_pages", torch.int32), dtype,
                                           num_layers, len(src_pools), ctypes.addressof(sp), src_pool_pages,
                                           len(recv_bufs), ctypes.addressof(rp),
                                           _dptr(dev_error, "dev_error", torch.int32), _stream(stream)),
           "dcp_naive_full_transfer")


def naive_inplace_shard(dst_vpages: torch.Tensor, num_layers: int, recv_bufs: list, dst_pools: list,
                        dst_slots_per_rank: int, dev_error: torch.Tensor | None = None, stream=None) -> None:
    """Baseline: each rank keeps the pages it owns from its full copy, at their DCP slots."""
    dtype = _kv_code(dst_pools[0])
    rp = _ptr_array(recv_bufs, "recv_bufs")
    dp = _ptr_array(dst_pools, "dst_pools")
    _check(_load().dcp_naive_inplace_shard(dst_vpages.numel(), _dptr(dst_vpages, "dst_vpages", torch.int32), dtype,
                                           num_layers, len(dst_pools), ctypes.addressof(rp), ctypes.addressof(dp),
                                           dst_slots_per_rank, _dptr(dev_error, "dev_error", torch.int32),
                                           _stream(stream)),
           "dcp_naive_inplace_shard")


def pack_chunks(n_items: int, page_bytes: int, staging_bytes: int) -> list:
    """Item ranges (begin, count) of a path's bounded pack: as many whole pages per chunk as the
    staging buffer holds; one chunk when everything fits."""
    per = staging_bytes // page_bytes
    if per < 1:
        raise ValueError("the staging buffer holds no page")
    return [(b, min(per, n_items - b)) for b in range(0, n_items, per)]


def pack_pages(src_idx: torch.Tensor, n_idx: int, n_layers: int, item_begin: int, n_items: int,
               src_pool: torch.Tensor, staging: torch.Tensor, dev_error: torch.Tensor | None = None,
               stream=None) -> None:
    """Bounded-pack send side of one path: items [item_begin, item_begin + n_items) (layer-major
    over the first n_idx entries of src_idx) from src_pool [n_layers][pages][64][576] into staging."""
    dtype = _kv_code(src_pool)
    _check(_load().dcp_pack_pages(n_idx, _dptr(src_idx, "src_idx", torch.int32), n_layers, item_begin, n_items,
                                  dtype, _dptr(src_pool, "src_pool"), src_pool.shape[1], _dptr(staging, "staging"),
                                  staging.numel() * staging.element_size(), _dptr(dev_error, "dev_error", torch.int32),
                                  _stream(stream)),
           "dcp_pack_pages")


def unpack_pages(dst_slot: torch.Tensor, n_idx: int, n_layers: int, layer_offset: int, item_begin: int,
                 n_items: int, staging: torch.Tensor, dst_pool: torch.Tensor, dev_error: torch.Tensor | None = None,
                 stream=None) -> None:
    """Bounded-pack receive side: the same items from staging into dst_pool
    [num_layers][slots][64][576] at layer layer_offset + j, slot dst_slot[i]."""
    dtype = _kv_code(dst_pool)
    _check(_load().dcp_unpack_pages(n_idx, _dptr(dst_slot, "dst_slot", torch.int32), n_layers, layer_offset,
                                    item_begin, n_items, dtype, _dptr(staging, "staging"),
                                    staging.numel() * staging.element_size(), _dptr(dst_pool, "dst_pool"),
                                    dst_pool.shape[0], dst_pool.shape[1], _dptr(dev_error, "dev_error", torch.int32),
                                    _stream(stream)),
           "dcp_unpack_pages")


def reshard_pages(req_page_ptr: torch.Tensor, src_pages: torch.Tensor, dst_vpages: torch.Tensor,
                  num_layers: int, src_pools: list, src_pool_pages: int, dst_pools: list,
                  dst_slots_per_rank: int, n_dcp: int | None = None, only_src_rank: int = -1,
                  only_dst_rank: int = -1, dev_error: torch.Tensor | None = None, stream=None) -> None:
    """Page-level reshard (all (r, d) paths in one launch); dst_pools are written in place."""
    dtype = _kv_code(src_pools[0])
    n_dcp = len(dst_pools) if n_dcp is None else n_dcp
    if n_dcp > len(dst_pools):
        raise ValueError(f"n_dcp = {n_dcp} but only {len(dst_pools)} destination pools")
    n_cp = len(src_pools)
    for r, p in enumerate(src_pools):
        lay, pages = _pool_pages(p, f"src_pools[{r}]")
        s0 = (num_layers // n_cp) * r + min(r, num_layers % n_cp)  # rank r's share of the layers
        need = num_layers // n_cp + (1 if r < num_layers % n_cp else 0)
        # the library addresses layer l of the pool at l * src_pool_pages pages
        if (p.dtype != src_pools[0].dtype or lay < need or src_pool_pages > pages
                or (need > 1 and src_pool_pages != pages)):
            raise ValueError(f"src_pools[{r}] must be [{need}][src_pool_pages = {src_pool_pages}][64][576] "
                             f"(layers from {s0}), got {tuple(p.shape)} {p.dtype}")
    for d, p in enumerate(dst_pools[:n_dcp]):
        lay, pages = _pool_pages(p, f"dst_pools[{d}]")
        if (p.dtype != src_pools[0].dtype or lay < num_layers or dst_slots_per_rank > pages
                or (num_layers > 1 and dst_slots_per_rank != pages)):
            raise ValueError(f"dst_pools[{d}] must be [{num_layers}][dst_slots_per_rank = {dst_slots_per_rank}]"
                             f"[64][576], got {tuple(p.shape)} {p.dtype}")
    sp = _ptr_array(src_pools, "src_pools")
    dp = _ptr_array(dst_pools, "dst_pools")
    _check(_load().dcp_reshard_pages(req_page_ptr.numel() - 1, _dptr(req_page_ptr, "req_page_ptr", torch.int64),
                                     dst_vpages.numel(), _dptr(src_pages, "src_pages", torch.int32),
                                     _dptr(dst_vpages, "dst_vpages", torch.int32), PAGE, K_DIM, dtype,
                                     num_layers, len(src_pools), ctypes.addressof(sp), src_pool_pages,
                                     n_dcp, ctypes.addressof(dp), dst_slots_per_rank, only_src_rank,
                                     only_dst_rank, _dptr(dev_error, "dev_error", torch.int32),
                                     _stream(stream)),
           "dcp_reshard_pages")


def _new(shape: tuple, dtype: torch.dtype, dev: torch.device, stream) -> torch.Tensor:
    """A new tensor for a call on `stream`: allocated on that stream, so that neither earlier work
    on its memory nor its later reuse overlaps the call."""
    if not isinstance(stream, torch.cuda.Stream):
        t = _views.empty(shape, dtype, dev.index) if _views else None
        return torch.empty(shape, dtype=dtype, device=dev) if t is None else t
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


# The checks of the calls below run once per call of a serving step, so they ask each tensor as
# little as possible: get_device() is -1 off the GPU and says "same device" and "on a GPU" at once.
def _device(t: torch.Tensor, name: str) -> int:
    """The index of a tensor's GPU, which must be the current one (the library launches there)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _raw_stream(stream, dev: int) -> int | None:
    return (torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream) or None


def _ptr(t: torch.Tensor | None, name: str, dtype: torch.dtype, dev: int) -> int | None:
    """Pointer of a contiguous tensor of this dtype on GPU `dev` (None for None)."""
    if t is None:
        return None
    p = _views.ptr(t, dtype, dev) if _views else None
    if p is not None:
        return p
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{dev}, got {t.dtype} on {t.device}")
    return t.data_ptr()


def _ptrs(tensors: list, name: str, like: torch.Tensor, dtype: torch.dtype, dev: int) -> bytes:
    """Host array of the pointers of tensors that all have this dtype and like's shape."""
    p = _views.ptrs(tensors, like, dtype, dev) if _views else None
    if p is not None:
        return p
    for t in tensors:
        if t.shape != like.shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"every tensor of {name} must be a contiguous {dtype} {tuple(like.shape)} on cuda:{dev}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return array("Q", [t.data_ptr() for t in tensors]).tobytes()


def _check_ptr(ptr: torch.Tensor, name: str) -> int:
    """Entries of a CSR offset array less one."""
    if ptr.dim() != 1 or ptr.numel() < 1:
        raise ValueError(f"{name} must be [requests + 1]")
    return ptr.numel() - 1


def _rows(t: torch.Tensor, name: str, width: int, dims: int, multiple: int, dev: int) -> tuple:
    """(pointer, outer strides...) of BF16 rows [..., width] whose last axis is contiguous and whose
    outer strides and start are multiples of `multiple` elements (strided views of wider rows are
    fine).  An axis of one entry may carry any stride: none is taken along it."""
    r = _views.rows(t, width, dims, multiple, dev) if _views else None
    if r is not None:
        return r
    shape, st = t.shape, t.stride()
    if len(shape) != dims or shape[-1] != width or t.dtype is not torch.bfloat16 or t.get_device() != dev:
        raise ValueError(f"{name} must be a bfloat16 tensor of {dims} axes, the last of {width}, on cuda:{dev}, "
                         f"got {t.dtype} {tuple(shape)} on {t.device}")
    p = t.data_ptr()
    s0 = st[0] if shape[0] > 1 else width
    s1 = multiple if dims == 2 else st[1] if shape[1] > 1 else width
    if (st[-1] != 1 and width > 1) or s0 % multiple or s1 % multiple or p % (2 * multiple):
        raise ValueError(f"{name}: the last axis must be contiguous, the other strides multiples of {multiple} and the start "
                         f"on a {2 * multiple}-byte boundary")
    return (p, s0) if dims == 2 else (p, s0, s1)


def _pools(kv_pools: list) -> torch.Size:
    """Shape [slots][64][576] of the pools (the others are compared with the first one's)."""
    if not kv_pools:
        raise ValueError("kv_pools is empty")
    shape = kv_pools[0].shape
    if len(shape) != 3 or shape[1] != PAGE or shape[2] != K_DIM:
        raise ValueError("every kv pool must be [slots][64][576] of one dtype")
    return shape


def _scale_block(kv_scales: list, kv_pools: list, slots: int, kv_scale: float) -> int:
    """Tokens per scale of block scales, per rank fp32 [slots][64 / block]."""
    if len(kv_scales) != len(kv_pools):
        raise ValueError("kv_scales must have one tensor per pool")
    if kv_pools[0].dtype is not torch.float8_e4m3fn:
        raise ValueError("kv_scales need float8_e4m3fn pools")
    if kv_scale != 1.0:
        raise ValueError("kv_scales stand in place of kv_scale, which must be 1")
    shape = kv_scales[0].shape
    if len(shape) != 2 or shape[0] != slots or not 1 <= shape[1] <= PAGE or PAGE % shape[1]:
        raise ValueError(f"kv_scales must be [{slots}][64 / block], block a power of two up to 64, got {tuple(shape)}")
    return PAGE // shape[1]


def append_kv(latent: torch.Tensor, rope: torch.Tensor, new_ptr: torch.Tensor, seq_lens: torch.Tensor,
              req_page_ptr: torch.Tensor, dst_vpages: torch.Tensor, kv_pools: list, inv_freq: torch.Tensor, *,
              rope_scale: float = 1.0, interleaved: bool = True, kv_scale: float = 1.0, kv_scales: list | None = None,
              q_rope: torch.Tensor | None = None, q_out: torch.Tensor | None = None, layout: str = "page",
              dev_error: torch.Tensor | None = None, stream=None) -> None:
    """New tokens' rows [latent 512 | rope 64] into kv_pools (in place): the rope part rotated by
    position * inv_freq (fp64 [32]), E4M3 pools quantised by kv_scale or by kv_scales (per rank
    [slots][64 / block], written too).  Request b's tokens are rows new_ptr[b] .. new_ptr[b + 1] - 1
    of latent [n][512] and rope [n][64] and its last positions below seq_lens[b].  q_rope
    [n][heads][64] is rotated alike into q_out, which may be q_rope.  See dcp_append_kv in dcp.h."""
    if layout != "page" and layout != "token":
        raise ValueError("layout must be 'page' or 'token'")
    dev = _device(latent, "latent")
    B = _check_ptr(new_ptr, "new_ptr")
    if seq_lens.numel() != B or req_page_ptr.numel() != B + 1:
        raise ValueError("new_ptr, seq_lens and req_page_ptr disagree on the number of requests")
    lp, ls = _rows(latent, "latent", V_DIM, 2, 8, dev)
    rp, rs = _rows(rope, "rope", K_DIM - V_DIM, 2, 2, dev)
    n = latent.shape[0]
    if rope.shape[0] != n:
        raise ValueError("latent and rope must have the same rows")
    shape = _pools(kv_pools)
    kind = kv_pools[0].dtype
    dtype = _kv_code(kv_pools[0])
    kp = _ptrs(kv_pools, "kv_pools", kv_pools[0], kind, dev)
    block, sp = 0, None
    if kv_scales is not None:
        block = _scale_block(kv_scales, kv_pools, shape[0], kv_scale)
        sp = _ptrs(kv_scales, "kv_scales", kv_scales[0], torch.float32, dev)
    if inv_freq.numel() != (K_DIM - V_DIM) // 2:
        raise ValueError("inv_freq must hold 32 values")
    heads, q, o = 0, (None, 0, 0), (None, 0, 0)
    if q_rope is not None or q_out is not None:
        if q_rope is None or q_out is None:
            raise ValueError("q_rope and q_out go together")
        q = _rows(q_rope, "q_rope", K_DIM - V_DIM, 3, 2, dev)
        o = _rows(q_out, "q_out", K_DIM - V_DIM, 3, 2, dev)
        heads = q_rope.shape[1]
        if q_rope.shape[0] != n or q_out.shape != q_rope.shape:
            raise ValueError("q_rope and q_out must be [rows of latent][heads][64]")
    st = _serving().dcp_append_kv(
        B, n, lp, ls, rp, rs, _ptr(new_ptr, "new_ptr", torch.int64, dev), _ptr(seq_lens, "seq_lens", torch.int32, dev),
        _ptr(req_page_ptr, "req_page_ptr", torch.int64, dev), dst_vpages.numel(),
        _ptr(dst_vpages, "dst_vpages", torch.int32, dev), PAGE, dtype, kv_scale, len(kv_pools), kp, shape[0], sp, block,
        _ptr(inv_freq, "inv_freq", torch.float64, dev), rope_scale, interleaved, layout == "token", heads, q[0], q[1], q[2],
        o[0], o[1], o[2], _ptr(dev_error, "dev_error", torch.int32, dev), _raw_stream(stream, dev))
    _check(st, "dcp_append_kv")


def reshard_scales(req_page_ptr: torch.Tensor, src_pages: torch.Tensor, dst_vpages: torch.Tensor, num_layers: int,
                   src_scales: list, dst_scales: list, dev_error: torch.Tensor | None = None, stream=None) -> None:
    """The block scales of reshard_pages' pages: src_scales per CP rank fp32 [layers of r][pages][64 / block],
    dst_scales per DCP rank [num_layers][slots][64 / block], written in place."""
    if not src_scales or not dst_scales:
        raise ValueError("src_scales and dst_scales must not be empty")
    dev = _device(dst_vpages, "dst_vpages")
    n_cp, n = len(src_scales), dst_vpages.numel()
    B = _check_ptr(req_page_ptr, "req_page_ptr")
    if src_pages.numel() != n:
        raise ValueError("src_pages and dst_vpages must have the same entries")
    src, dst = src_scales[0].shape, dst_scales[0].shape
    if len(src) != 3 or len(dst) != 3 or dst[0] != num_layers or dst[2] != src[2] or not 1 <= src[2] <= PAGE or PAGE % src[2]:
        raise ValueError("scales must be [layers][pages][64 / block], block a power of two up to 64; dst_scales of every layer")
    pages, groups = src[1], src[2]
    # the ranks below num_layers mod n_cp hold one layer more (dcp_layer_range)
    more = num_layers % n_cp
    low = num_layers // n_cp
    if src[0] != low + (more > 0) or (0 < more and tuple(src_scales[more].shape) != (low, pages, groups)):
        raise ValueError(f"src_scales must hold their ranks' layers of {num_layers}, [{pages}][{groups}] each")
    sp = (_ptrs(src_scales[:more], "src_scales", src_scales[0], torch.float32, dev)
          + _ptrs(src_scales[more:], "src_scales", src_scales[more], torch.float32, dev))
    dp = _ptrs(dst_scales, "dst_scales", dst_scales[0], torch.float32, dev)
    _check(_serving().dcp_reshard_scales(
        B, _ptr(req_page_ptr, "req_page_ptr", torch.int64, dev), n, _ptr(src_pages, "src_pages", torch.int32, dev),
        _ptr(dst_vpages, "dst_vpages", torch.int32, dev), PAGE // groups, num_layers, n_cp, sp, pages, len(dst_scales), dp, dst[1],
        _ptr(dev_error, "dev_error", torch.int32, dev), _raw_stream(stream, dev)),
           "dcp_reshard_scales")


def workspace_size(num_requests: int, q_len: int, num_heads: int, n_dcp: int, num_pages: int) -> int:
    return int(_serving().dcp_partial_decode_attn_workspace_size(num_requests, q_len, num_heads, n_dcp, num_pages))


def _workspace_bytes(num_requests: int, q_len: int, num_heads: int, n_dcp: int, num_pages: int) -> int:
    n = workspace_size(num_requests, q_len, num_heads, n_dcp, num_pages)
    if n == 0:
        raise DcpError(-1, "dcp_partial_decode_attn_workspace_size")
    return n


def alloc_workspace(num_requests: int, q_len: int, num_heads: int, n_dcp: int, num_pages: int,
                    device) -> torch.Tensor:
    return torch.empty(_workspace_bytes(num_requests, q_len, num_heads, n_dcp, num_pages), dtype=torch.uint8, device=device)


def partial_decode_attn(q: torch.Tensor, seq_lens: torch.Tensor, req_page_ptr: torch.Tensor,
                        dst_vpages: torch.Tensor, kv_pools: list, softmax_scale: float,
                        kv_scale: float = 1.0, only_rank: int = -1, o_part: torch.Tensor | None = None,
                        lse_part: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        dev_error: torch.Tensor | None = None, stream=None, layout: str = "page",
                        planned: bool = False, kv_scales: list | None = None):
    """Per-rank partial attention.  q: bf16 [B][T][H][576]; kv_pools: per-rank [slots][64][576].
    layout "token": the page table is token-interleaved (dcp_partial_decode_attn_tokens).
    planned: run the plan attn_plan stored in ``workspace`` (dcp_partial_decode_attn_run).
    kv_scales: block scales of E4M3 pools, per rank fp32 [slots][64 / block], in place of kv_scale
    (dcp_partial_decode_attn_scaled).
    Returns (o_part [N][B][T][H][512] fp32, lse_part [N][B][T][H] fp32)."""
    B, T, H, kd = q.shape
    if kd != K_DIM:
        raise ValueError("q must be [B][T][H][576]")
    _check_table(B, seq_lens, req_page_ptr)
    N = len(kv_pools)
    slots, dtype = _check_pools(kv_pools)
    _check_out(o_part, (N, B, T, H, V_DIM), "o_part")
    _check_out(lse_part, (N, B, T, H), "lse_part")
    dev = q.device
    if planned and (layout == "token" or workspace is None):
        raise ValueError("a planned run needs the workspace holding the plan (page layout)")
    if kv_scales is not None:
        _device(q, "q")
        block = _scale_block(kv_scales, kv_pools, slots, kv_scale)
    if o_part is None:
        o_part = _new((N, B, T, H, V_DIM), torch.float32, dev, stream)
    if lse_part is None:
        lse_part = _new((N, B, T, H), torch.float32, dev, stream)
    num_pages = dst_vpages.numel()
    if workspace is None:
        workspace = _new((_workspace_bytes(B, T, H, N, num_pages),), torch.uint8, dev, stream)
    if kv_scales is not None:
        if layout not in ("page", "token"):
            raise ValueError("layout must be 'page' or 'token'")
        d = q.get_device()
        kp = _ptrs(kv_pools, "kv_pools", kv_pools[0], torch.float8_e4m3fn, d)
        sp = _ptrs(kv_scales, "kv_scales", kv_scales[0], torch.float32, d)
        _check(_serving().dcp_partial_decode_attn_scaled(
            B, T, H, _ptr(q, "q", torch.bfloat16, d), _ptr(seq_lens, "seq_lens", torch.int32, d),
            _ptr(req_page_ptr, "req_page_ptr", torch.int64, d), num_pages, _ptr(dst_vpages, "dst_vpages", torch.int32, d), PAGE,
            softmax_scale, N, kp, slots, sp, block, only_rank, _ptr(o_part, "o_part", torch.float32, d),
            _ptr(lse_part, "lse_part", torch.float32, d), _ptr(workspace, "workspace", torch.uint8, d), workspace.numel(),
            layout == "token", planned, _ptr(dev_error, "dev_error", torch.int32, d), _raw_stream(stream, d)),
               "dcp_partial_decode_attn_scaled")
        return o_part, lse_part
    kp = _ptr_array(kv_pools, "kv_pools")
    fn = (_load().dcp_partial_decode_attn_run if planned else
          _load().dcp_partial_decode_attn_tokens if layout == "token" else _load().dcp_partial_decode_attn)
    _check(fn(B, T, H, _dptr(q, "q", torch.bfloat16),
                                           _dptr(seq_lens, "seq_lens", torch.int32),
                                           _dptr(req_page_ptr, "req_page_ptr", torch.int64), num_pages,
                                           _dptr(dst_vpages, "dst_vpages", torch.int32), PAGE, dtype,
                                           float(kv_scale), float(softmax_scale), N, ctypes.addressof(kp),
                                           slots, only_rank, _dptr(o_part, "o_part", torch.float32),
                                           _dptr(lse_part, "lse_part", torch.float32),
                                           _dptr(workspace, "workspace"), workspace.numel(),
                                           _dptr(dev_error, "dev_error", torch.int32), _stream(stream)),
           "dcp_partial_decode_attn")
    return o_part, lse_part


def attn_plan(q_shape: tuple, req_page_ptr: torch.Tensor, dst_vpages: torch.Tensor, kv_pools: list,
              workspace: torch.Tensor, only_rank: int = -1, dev_error: torch.Tensor | None = None, stream=None) -> None:
    """The attention's plan for this page table into ``workspace`` (dcp_attn_plan); q_shape =
    (B, T, H); kv_pools give the DCP size, slots per rank and dtype."""
    B, T, H = q_shape[:3]
    _check_table(B, None, req_page_ptr)
    _check_pools(kv_pools)
    _check(_load().dcp_attn_plan(B, T, H, _dptr(req_page_ptr, "req_page_ptr", torch.int64), dst_vpages.numel(),
                                 _dptr(dst_vpages, "dst_vpages", torch.int32), _kv_code(kv_pools[0]), len(kv_pools),
                                 kv_pools[0].shape[0], only_rank, _dptr(workspace, "workspace"), workspace.numel(),
                                 _dptr(dev_error, "dev_error", torch.int32), _stream(stream)),
           "dcp_attn_plan")


def attn_plan_info(q_shape: tuple, num_pages: int, kv_pools: list, workspace: torch.Tensor, stream=None) -> dict:
    """The header of the plan in ``workspace`` (dcp_attn_plan_info, synchronous): work units in
    the queue, (rank, request) pairs split into several pieces, tiles per chunk, and whether the
    workspace holds a plan at all."""
    B, T, H = q_shape[:3]
    _check_pools(kv_pools)
    info = (ctypes.c_int32 * 4)()
    _check(_load().dcp_attn_plan_info(B, T, H, int(num_pages), _kv_code(kv_pools[0]), len(kv_pools),
                                      _dptr(workspace, "workspace"), workspace.numel(), ctypes.addressof(info),
                                      _stream(stream)),
           "dcp_attn_plan_info")
    return {"units": info[0], "split_pairs": info[1], "tiles_per_chunk": info[2], "valid": bool(info[3])}


def _merged_scaled(q, seq_lens, req_page_ptr, dst_vpages, kv_pools, softmax_scale, kv_scale, o_part, lse_part, o_out, lse_out,
                   workspace, dev_error, stream, planned, layout, kv_scales, o_dtype):
    """decode_attn_merged with block scales or a BF16 output (its outputs' shapes are checked)."""
    B, T, H, _ = q.shape
    N, d, num_pages = len(kv_pools), _device(q, "q"), dst_vpages.numel()
    shape = _pools(kv_pools)
    kind, code = kv_pools[0].dtype, _kv_code(kv_pools[0])
    kp = _ptrs(kv_pools, "kv_pools", kv_pools[0], kind, d)
    block, sp = 0, None
    if kv_scales is not None:
        block = _scale_block(kv_scales, kv_pools, shape[0], kv_scale)
        sp = _ptrs(kv_scales, "kv_scales", kv_scales[0], torch.float32, d)
    dev = q.device
    if o_part is None:
        o_part = _new((N, B, T, H, V_DIM), torch.float32, dev, stream)
    if lse_part is None:
        lse_part = _new((N, B, T, H), torch.float32, dev, stream)
    if o_out is None:
        o_out = _new((B, T, H, V_DIM), o_dtype, dev, stream)
    if lse_out is None:
        lse_out = _new((B, T, H), torch.float32, dev, stream)
    if workspace is None:
        workspace = _new((_workspace_bytes(B, T, H, N, num_pages),), torch.uint8, dev, stream)
    _check(_serving().dcp_decode_attn_merged_scaled(
        B, T, H, _ptr(q, "q", torch.bfloat16, d), _ptr(seq_lens, "seq_lens", torch.int32, d),
        _ptr(req_page_ptr, "req_page_ptr", torch.int64, d), num_pages, _ptr(dst_vpages, "dst_vpages", torch.int32, d), PAGE,
        code, kv_scale, softmax_scale, N, kp, shape[0], sp, block, _ptr(o_part, "o_part", torch.float32, d),
        _ptr(lse_part, "lse_part", torch.float32, d), _ptr(o_out, "o_out", o_dtype, d), o_dtype is torch.bfloat16,
        _ptr(lse_out, "lse_out", torch.float32, d), _ptr(workspace, "workspace", torch.uint8, d), workspace.numel(),
        layout == "token", planned, _ptr(dev_error, "dev_error", torch.int32, d), _raw_stream(stream, d)),
           "dcp_decode_attn_merged_scaled")
    return o_out, lse_out, o_part, lse_part


def decode_attn_merged(q: torch.Tensor, seq_lens: torch.Tensor, req_page_ptr: torch.Tensor,
                       dst_vpages: torch.Tensor, kv_pools: list, softmax_scale: float, kv_scale: float = 1.0,
                       o_part: torch.Tensor | None = None, lse_part: torch.Tensor | None = None,
                       o_out: torch.Tensor | None = None, lse_out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, dev_error: torch.Tensor | None = None, stream=None,
                       planned: bool = False, layout: str = "page", kv_scales: list | None = None,
                       o_dtype: torch.dtype = torch.float32):
    """Every rank's partial attention plus their exact LSE merge in one call (planned: run the
    plan attn_plan stored in ``workspace``, dcp_decode_attn_merged_run; layout "token": the page
    table is token-interleaved, dcp_decode_attn_merged_tokens; kv_scales: block scales of E4M3
    pools in place of kv_scale, dcp_decode_attn_merged_scaled).
    Returns (o_out [B][T][H][512] of o_dtype, float32 or bfloat16, lse_out [B][T][H], o_part,
    lse_part), the others fp32."""
    if layout not in ("page", "token"):
        raise ValueError("layout must be 'page' or 'token'")
    if planned and (workspace is None or layout == "token"):
        raise ValueError("a planned run needs the workspace holding the plan (page layout)")
    B, T, H, kd = q.shape
    if kd != K_DIM:
        raise ValueError("q must be [B][T][H][576]")
    _check_table(B, seq_lens, req_page_ptr)
    N = len(kv_pools)
    _check_out(o_part, (N, B, T, H, V_DIM), "o_part")
    _check_out(lse_part, (N, B, T, H), "lse_part")
    if o_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("o_dtype must be float32 or bfloat16")
    if o_out is not None and (tuple(o_out.shape) != (B, T, H, V_DIM) or o_out.dtype != o_dtype):
        raise ValueError(f"o_out must be {o_dtype} {(B, T, H, V_DIM)}, got {o_out.dtype} {tuple(o_out.shape)}")
    _check_out(lse_out, (B, T, H), "lse_out")
    if kv_scales is not None or o_dtype is not torch.float32:
        return _merged_scaled(q, seq_lens, req_page_ptr, dst_vpages, kv_pools, softmax_scale, kv_scale, o_part, lse_part, o_out,
                              lse_out, workspace, dev_error, stream, planned, layout, kv_scales, o_dtype)
    slots, dtype = _check_pools(kv_pools)
    dev = q.device
    if o_part is None:
        o_part = _new((N, B, T, H, V_DIM), torch.float32, dev, stream)
    if lse_part is None:
        lse_part = _new((N, B, T, H), torch.float32, dev, stream)
    if o_out is None:
        o_out = _new((B, T, H, V_DIM), o_dtype, dev, stream)
    if lse_out is None:
        lse_out = _new((B, T, H), torch.float32, dev, stream)
    num_pages = dst_vpages.numel()
    if workspace is None:
        workspace = _new((_workspace_bytes(B, T, H, N, num_pages),), torch.uint8, dev, stream)
    kp = _ptr_array(kv_pools, "kv_pools")
    fn = (_load().dcp_decode_attn_merged_run if planned else
          _load().dcp_decode_attn_merged_tokens if layout == "token" else _load().dcp_decode_attn_merged)
    _check(fn(B, T, H, _dptr(q, "q", torch.bfloat16),
                                          _dptr(seq_lens, "seq_lens", torch.int32),
                                          _dptr(req_page_ptr, "req_page_ptr", torch.int64), num_pages,
                                          _dptr(dst_vpages, "dst_vpages", torch.int32), PAGE, dtype,
                                          float(kv_scale), float(softmax_scale), N, ctypes.addressof(kp), slots,
                                          _dptr(o_part, "o_part", torch.float32),
                                          _dptr(lse_part, "lse_part", torch.float32),
                                          _dptr(o_out, "o_out", torch.float32),
                                          _dptr(lse_out, "lse_out", torch.float32),
                                          _dptr(workspace, "workspace"), workspace.numel(),
                                          _dptr(dev_error, "dev_error", torch.int32), _stream(stream)),
           "dcp_decode_attn_merged")
    return o_out, lse_out, o_part, lse_part


def partial_decode_attn_static(q: torch.Tensor, seq_lens: torch.Tensor, req_page_ptr: torch.Tensor,
                               dst_vpages: torch.Tensor, kv_pools: list, softmax_scale: float,
                               kv_scale: float = 1.0, only_rank: int = -1, o_part: torch.Tensor | None = None,
                               lse_part: torch.Tensor | None = None, dev_error: torch.Tensor | None = None,
                               stream=None):
    """Same as partial_decode_attn, for callers that cannot allocate device memory: the call
    uses the library's fixed device scratch array instead of a workspace.  The outputs must be
    passed in by such callers (they are only allocated here when omitted, for convenience)."""
    B, T, H, kd = q.shape
    if kd != K_DIM:
        raise ValueError("q must be [B][T][H][576]")
    _check_table(B, seq_lens, req_page_ptr)
    N = len(kv_pools)
    slots, dtype = _check_pools(kv_pools)
    _check_out(o_part, (N, B, T, H, V_DIM), "o_part")
    _check_out(lse_part, (N, B, T, H), "lse_part")
    dev = q.device
    if o_part is None:
        o_part = torch.empty((N, B, T, H, V_DIM), dtype=torch.float32, device=dev)
    if lse_part is None:
        lse_part = torch.empty((N, B, T, H), dtype=torch.float32, device=dev)
    kp = _ptr_array(kv_pools, "kv_pools")
    _check(_load().dcp_partial_decode_attn_static(B, T, H, _dptr(q, "q", torch.bfloat16),
                                                  _dptr(seq_lens, "seq_lens", torch.int32),
                                                  _dptr(req_page_ptr, "req_page_ptr", torch.int64),
                                                  dst_vpages.numel(), _dptr(dst_vpages, "dst_vpages", torch.int32),
                                                  PAGE, dtype, float(kv_scale), float(softmax_scale), N,
                                                  ctypes.addressof(kp), slots, only_rank,
                                                  _dptr(o_part, "o_part", torch.float32),
                                                  _dptr(lse_part, "lse_part", torch.float32),
                                                  _dptr(dev_error, "dev_error", torch.int32), _stream(stream)),
           "dcp_partial_decode_attn_static")
    return o_part, lse_part


def lse_merge(o_part: torch.Tensor, lse_part: torch.Tensor, o_out: torch.Tensor | None = None,
              lse_out: torch.Tensor | None = None, stream=None):
    """Merge [N][rows...][v] partials into [rows...][v]; returns (o, lse)."""
    n = o_part.shape[0]
    v = o_part.shape[-1]
    rows = lse_part[0].numel()
    if o_part.numel() != n * rows * v:
        raise ValueError("o_part / lse_part shapes disagree")
    for t, want, name in ((o_out, rows * v, "o_out"), (lse_out, rows, "lse_out")):
        if t is not None and (t.numel() != want or t.dtype != torch.float32):
            raise ValueError(f"{name} must be float32 with {want} elements")
    if o_out is None:
        o_out = torch.empty(o_part.shape[1:], dtype=torch.float32, device=o_part.device)
    if lse_out is None:
        lse_out = torch.empty(lse_part.shape[1:], dtype=torch.float32, device=o_part.device)
    _check(_load().dcp_lse_merge(n, rows, v, _dptr(o_part, "o_part", torch.float32),
                                 _dptr(lse_part, "lse_part", torch.float32),
                                 _dptr(o_out, "o_out", torch.float32), _dptr(lse_out, "lse_out", torch.float32),
                                 _stream(stream)),
           "dcp_lse_merge")
    return o_out, lse_out


def prefill_attn(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, q_ptr: torch.Tensor,
                 k_ptr: torch.Tensor, softmax_scale: float, causal: bool = True, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                 workspace: torch.Tensor | None = None, dev_error: torch.Tensor | None = None, stream=None):
    """Expanded latent attention of packed prompts.  q bf16 [n_q][H][192], k_nope [n_k][H][128], k_rope [n_k][64]
    (shared by the heads), v [n_k][H][128] (strided views of wider rows are fine); q_ptr, k_ptr int64 [B + 1].  causal:
    a request's queries are the last tokens of its keys.  Returns (out [n_q][H][128] of out_dtype, bfloat16 or
    float32, lse fp32 [n_q][H]).  See dcp_prefill_attn in dcp.h."""
    dev = _device(q, "q")
    B = _check_ptr(q_ptr, "q_ptr")
    if k_ptr.dim() != 1 or k_ptr.numel() != B + 1:
        raise ValueError("q_ptr and k_ptr disagree on the number of requests")
    qp, qt, qh = _rows(q, "q", 192, 3, 8, dev)
    kp, kt, kh = _rows(k_nope, "k_nope", 128, 3, 8, dev)
    vp, vt, vh = _rows(v, "v", 128, 3, 8, dev)
    rp, rt = _rows(k_rope, "k_rope", 64, 2, 8, dev)
    n_q, H, _ = q.shape
    n_k = k_nope.shape[0]
    if k_nope.shape[1] != H or v.shape != k_nope.shape or k_rope.shape[0] != n_k or H < 1:
        raise ValueError("q, k_nope, k_rope and v disagree on heads or key rows")
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is None:
        out = _new((n_q, H, 128), out_dtype, q.device, stream)
    elif out.shape != (n_q, H, 128):
        raise ValueError(f"out must be {(n_q, H, 128)}, got {tuple(out.shape)}")
    if lse is None:
        lse = _new((n_q, H), torch.float32, q.device, stream)
    elif lse.shape != (n_q, H):
        raise ValueError(f"lse must be {(n_q, H)}, got {tuple(lse.shape)}")
    lib = _serving()
    need = lib.dcp_prefill_attn_workspace_size(B, n_q, n_k, H)
    if need and workspace is None:
        workspace = _new((need,), torch.uint8, q.device, stream)
    _check(lib.dcp_prefill_attn(
        B, n_q, n_k, H, qp, qt, qh, kp, kt, kh, rp, rt, vp, vt, vh, _ptr(q_ptr, "q_ptr", torch.int64, dev),
        _ptr(k_ptr, "k_ptr", torch.int64, dev), softmax_scale, bool(causal), _ptr(out, "out", out_dtype, dev),
        out_dtype is torch.bfloat16, _ptr(lse, "lse", torch.float32, dev), _ptr(workspace, "workspace", torch.uint8, dev),
        workspace.numel() if workspace is not None else 0, _ptr(dev_error, "dev_error", torch.int32, dev), _raw_stream(stream, dev)),
           "dcp_prefill_attn")
    return out, lse


def selftest_wait_timeout(limit_ns: int, dev_error: torch.Tensor, out_ok: torch.Tensor, stream=None) -> None:
    """Run the library's bounded pipeline wait on a barrier nothing completes (see dcp.h):
    afterwards dev_error has DEVERR_TIMEOUT set and out_ok holds 0."""
    _check(_load().dcp_selftest_wait_timeout(int(limit_ns), _dptr(dev_error, "dev_error", torch.int32),
                                             _dptr(out_ok, "out_ok", torch.int32), _stream(stream)),
           "dcp_selftest_wait_timeout")
