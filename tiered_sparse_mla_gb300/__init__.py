"""GB300 (sm_103a) tiered sparse-MLA decode path: Python binding of ``include/hs.h``.

Thin ctypes marshalling over ``libhs.so``: every step of the path runs in the
library's CUDA kernels. PyTorch supplies device memory (tensor data pointers)
and streams only. Function names follow the C ABI (``hs_pool_create``,
``hs_resolve_topk``, ``hs_sparse_mla_decode`` ...); :class:`Pool` is a small
convenience wrapper around a pool handle.

There is no CPU fallback: importing the ops without a built library, or using
them on a device other than sm_103, raises.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhs.so")

HS_OK, HS_ERR_INVALID_ARG, HS_ERR_CAPACITY, HS_ERR_OUT_OF_MEMORY = 0, 1, 2, 3
HS_ERR_CUDA, HS_ERR_DEVICE_DATA, HS_ERR_TIMEOUT, HS_ERR_UNSUPPORTED = 4, 5, 6, 7
HS_DEVERR_INDEX_RANGE, HS_DEVERR_DUPLICATE, HS_DEVERR_NO_HOST = 1, 2, 4
HS_DEVERR_BAD_REQUEST, HS_DEVERR_CAPACITY, HS_DEVERR_TIMEOUT = 8, 16, 32
HS_DEVERR_BAD_PAGE = 64
HS_BF16, HS_FP8_E4M3_ROWSCALE = 0, 1
HS_EVICT_SAVED_ONLY, HS_EVICT_PLAN = 1, 2
HS_PROB_F32, HS_PROB_BF16 = 0, 1

EXPORTED = [
    "hs_pool_create", "hs_pool_destroy", "hs_pool_get_config", "hs_pool_get_tables",
    "hs_request_init", "hs_request_set_ctx_len", "hs_set_ctx_len", "hs_page_map",
    "hs_page_map_range", "hs_hot_lease", "hs_hot_release", "hs_gpu_rows", "hs_host_rows",
    "hs_gpu_scales", "hs_host_scales", "hs_host_rows_device", "hs_host_scales_device",
    "hs_pool_snapshot", "hs_pool_restore",
    "hs_pool_get_error", "hs_resolve_topk", "hs_sparse_mla_decode",
    "hs_decode_workspace_bytes", "hs_status_string", "hs_sparse_mla_decode_static_ws",
    "hs_pool_check_bounded_wait", "hs_resolve_topk_union", "hs_sparse_mla_decode_per_token",
    "hs_layer_group_create", "hs_layer_group_destroy", "hs_resolve_topk_layers",
    "hs_active_copy", "hs_demote_cold_pages", "hs_append_rows", "hs_page_means",
    "hs_select_pages", "hs_select_workspace_bytes", "hs_page_mla_decode",
    "hs_page_decode_workspace_bytes", "hs_page_mla_decode_per_token",
    "hs_page_mla_decode_window", "hs_window_workspace_bytes", "hs_page_weights",
    "hs_weights_workspace_bytes", "hs_evict_pages", "hs_verify_drafts",
]
HS_STATIC_DECODE_WS_BYTES = 24 << 20


class HsError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


class hs_pool_config(C.Structure):
    _fields_ = [("nope_dim", C.c_int32), ("rope_dim", C.c_int32), ("page_size", C.c_int32),
                ("dtype", C.c_int32), ("n_gpu_blocks", C.c_int64), ("n_host_blocks", C.c_int64),
                ("max_requests", C.c_int32), ("max_ctx", C.c_int32), ("hot_rows", C.c_int32),
                ("max_topk", C.c_int32)]


class hs_pool_tables(C.Structure):
    _fields_ = [("page_table", C.c_void_p), ("hot_blocks", C.c_void_p), ("slot_tag", C.c_void_p),
                ("slot_stamp", C.c_void_p), ("lru_order", C.c_void_p),
                ("pos_to_slot", C.c_void_p), ("clock", C.c_void_p), ("ctx_len", C.c_void_p),
                ("max_pages", C.c_int32), ("row_bytes", C.c_int32)]


_lib = None


def load() -> C.CDLL:
    """Loads libhs.so. Raises if it was not built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            "tiered_sparse_mla_gb300: libhs.so is not built; run "
            "`python -c 'import __graft_entry__ as g; g.build()'` first")
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    sig = {
        "hs_pool_create": ([C.POINTER(hs_pool_config), vp, C.POINTER(vp)], i32),
        "hs_pool_destroy": ([vp], i32),
        "hs_pool_get_config": ([vp, C.POINTER(hs_pool_config)], i32),
        "hs_pool_get_tables": ([vp, C.POINTER(hs_pool_tables)], i32),
        "hs_request_init": ([vp, i32, i32], i32),
        "hs_request_set_ctx_len": ([vp, i32, i32], i32),
        "hs_set_ctx_len": ([vp, vp, i32, vp], i32),
        "hs_page_map": ([vp, i32, i32, i64, i64], i32),
        "hs_page_map_range": ([vp, i32, i32, i32, vp, vp], i32),
        "hs_hot_lease": ([vp, i32, vp, i32], i32),
        "hs_hot_release": ([vp, i32], i32),
        "hs_gpu_rows": ([vp], vp), "hs_host_rows": ([vp], vp),
        "hs_gpu_scales": ([vp], vp), "hs_host_scales": ([vp], vp),
        "hs_host_rows_device": ([vp], vp), "hs_host_scales_device": ([vp], vp),
        "hs_pool_snapshot": ([vp, vp, sz, C.POINTER(sz)], i32),
        "hs_pool_restore": ([vp, vp, sz], i32),
        "hs_pool_get_error": ([vp, C.POINTER(C.c_uint32)], i32),
        "hs_resolve_topk": ([vp, i32, vp, vp, i32, vp, vp, vp, vp, vp], i32),
        "hs_sparse_mla_decode": ([vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, C.c_float,
                                  vp, vp, vp, sz, vp], i32),
        "hs_decode_workspace_bytes": ([i32, i32, i32, i32], sz),
        "hs_sparse_mla_decode_static_ws": ([vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp,
                                            C.c_float, vp, vp, vp], i32),
        "hs_status_string": ([i32], C.c_char_p),
        "hs_resolve_topk_union": ([vp, i32, vp, vp, i32, vp, vp, vp, vp, vp], i32),
        "hs_layer_group_create": ([C.POINTER(vp), i32, C.POINTER(vp)], i32),
        "hs_layer_group_destroy": ([vp], i32),
        "hs_resolve_topk_layers": ([vp, i32, vp, vp, i32, vp, vp, vp, vp, vp], i32),
        "hs_active_copy": ([vp, i32, vp, vp, vp, vp], i32),
        "hs_demote_cold_pages": ([vp, i32, vp, vp, vp, vp, vp], i32),
        "hs_sparse_mla_decode_per_token": ([vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp,
                                            C.c_float, vp, vp, vp, sz, vp], i32),
        "hs_pool_check_bounded_wait": ([vp, C.c_uint32, vp], i32),
        "hs_append_rows": ([vp, i32, i32, vp, vp, vp, vp, vp], i32),
        "hs_page_means": ([vp, i32, vp, vp, vp, vp], i32),
        "hs_select_pages": ([vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz,
                             vp], i32),
        "hs_select_workspace_bytes": ([vp, i32, i32], sz),
        "hs_page_mla_decode": ([vp, i32, i32, i32, i32, vp, vp, vp, vp, C.c_float, vp, vp, vp,
                                sz, vp], i32),
        "hs_page_decode_workspace_bytes": ([i32, i32, i32, i32], sz),
        "hs_page_mla_decode_per_token": ([vp, i32, i32, i32, i32, vp, vp, vp, vp, C.c_float, vp,
                                          vp, vp, sz, vp], i32),
        "hs_page_mla_decode_window": ([vp, i32, i32, i32, i32, i32, vp, vp, vp, C.c_float, vp, vp,
                                       vp, sz, vp], i32),
        "hs_window_workspace_bytes": ([vp, i32, i32, i32, i32, i32], sz),
        "hs_page_weights": ([vp, i32, i32, i32, vp, vp, vp, vp, C.c_float, C.c_float, vp, vp, vp,
                             sz, vp], i32),
        "hs_weights_workspace_bytes": ([vp, i32, i32, i32], sz),
        "hs_evict_pages": ([vp, i32, i32, i32, i32, C.c_uint32, vp, vp, vp, vp, vp, vp, vp], i32),
        "hs_verify_drafts": ([vp, i32, i32, i32, i32, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp,
                              vp], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().hs_status_string(status).decode()


def _check(fn: str, st: int):
    if st != HS_OK:
        raise HsError(fn, st)


def _ptr(t) -> int | None:
    """Device pointer of a CUDA tensor (None passes NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _arg(name: str, t, dtype: str, *shape, optional: bool = False) -> int | None:
    """Device pointer of a CUDA tensor whose type (a torch dtype's name) and shape
    are checked first: the kernels read it by both."""
    if t is None and optional:
        return None
    # one look at a tensor that is as it should be: a call takes a few microseconds
    try:
        if (t.shape == shape and t.dtype is _dtypes[dtype] and t.get_device() == _only_device
                and t.is_contiguous()):
            return t.data_ptr()
    except (AttributeError, KeyError):
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a CUDA tensor")
    _dtypes[dtype] = getattr(torch, dtype)
    if t.dtype is not _dtypes[dtype]:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")
    return _here(name, t)


_dtypes: dict = {}
_only_device = None  # 0 once seen that the process has one CUDA device


def _here(name: str, t) -> int:
    """Device pointer of a contiguous tensor on the current CUDA device (the library
    refuses a pool of another one)."""
    import torch
    global _only_device
    p, dev = _ptr(t), torch.cuda.current_device()
    if t.get_device() != dev:
        raise ValueError(f"{name}: on CUDA device {t.get_device()}, the current one is {dev}")
    if torch.cuda.device_count() == 1:
        _only_device = 0
    return p


def _ws(workspace):
    if workspace is None:
        return 0, None
    n = workspace.numel() * workspace.element_size()
    if workspace.get_device() == _only_device and workspace.is_contiguous():
        return n, workspace.data_ptr()
    return n, _here("workspace", workspace)


_raw_stream = None


def _stream(stream) -> int | None:
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            # the current stream's handle, without a Stream object for it
            get_dev = getattr(torch._C, "_cuda_getDevice", None)
            get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            if get is None or get_dev is None or not torch.cuda.is_initialized():
                return torch.cuda.current_stream().cuda_stream
            _raw_stream = lambda: get(get_dev())
        return _raw_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


class _CudaArray:
    def __init__(self, ptr: int, shape, typestr: str, owner):
        self.owner = owner  # a tensor over the pool's memory keeps the pool
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (ptr, False), "version": 3, "strides": None}


def _device_view(ptr: int, shape, typestr: str, owner=None):
    import torch
    return torch.as_tensor(_CudaArray(ptr, shape, typestr, owner), device="cuda")


# ------------------------------------------------------------- C ABI functions
def hs_pool_create(cfg: hs_pool_config, stream=None) -> int:
    h = C.c_void_p()
    _check("hs_pool_create", load().hs_pool_create(C.byref(cfg), _stream(stream), C.byref(h)))
    return h.value


def hs_pool_destroy(pool: int):
    _check("hs_pool_destroy", load().hs_pool_destroy(pool))


def hs_resolve_topk(pool: int, req_ids, topk_idx, resolved, gathered, gathered_scale, counts,
                    stream=None):
    """One decode step's resolve (see hs.h). Tensors: req_ids int32 [B], topk_idx
    int32 [B][K], resolved int32 [B][K], gathered uint8 [B][K][row_bytes],
    gathered_scale float32 [B][K] or None, counts int32 [B][3]."""
    B, K = topk_idx.shape
    _check("hs_resolve_topk", load().hs_resolve_topk(
        pool, B, _ptr(req_ids), _ptr(topk_idx), K, _ptr(resolved), _ptr(gathered),
        _ptr(gathered_scale), _ptr(counts), _stream(stream)))


def hs_resolve_topk_union(pool: int, req_ids, topk_idx, resolved, gathered, gathered_scale,
                          counts, stream=None):
    """Resolve of several lists per request as their union (see hs.h). topk_idx
    int32 [B][T*K] (or [B][T][K]): each request's tokens' lists, concatenated;
    other tensors as hs_resolve_topk with K replaced by T*K."""
    B = topk_idx.shape[0]
    K = topk_idx.numel() // max(B, 1)
    _check("hs_resolve_topk_union", load().hs_resolve_topk_union(
        pool, B, _ptr(req_ids), _ptr(topk_idx), K, _ptr(resolved), _ptr(gathered),
        _ptr(gathered_scale), _ptr(counts), _stream(stream)))


def hs_layer_group_create(pools) -> int:
    """Group of pools (one per layer) for hs_resolve_topk_layers; returns a handle."""
    arr = (C.c_void_p * len(pools))(*[p.handle if hasattr(p, "handle") else p for p in pools])
    h = C.c_void_p()
    _check("hs_layer_group_create", load().hs_layer_group_create(arr, len(pools), C.byref(h)))
    return h.value


def hs_layer_group_destroy(group: int):
    _check("hs_layer_group_destroy", load().hs_layer_group_destroy(group))


def hs_resolve_topk_layers(group: int, req_ids, topk_idx, resolved, gathered, gathered_scale,
                           counts, stream=None):
    """All layers' resolve in one launch (see hs.h). topk_idx / resolved int32
    [L][B][K]; gathered [L][B][K][row_bytes] or None; gathered_scale [L][B][K]
    or None; counts int32 [L][B][3]."""
    _, B, K = topk_idx.shape
    _check("hs_resolve_topk_layers", load().hs_resolve_topk_layers(
        group, B, _ptr(req_ids), _ptr(topk_idx), K, _ptr(resolved), _ptr(gathered),
        _ptr(gathered_scale), _ptr(counts), _stream(stream)))


def hs_active_copy(pool: int, req, page, host_block, stream=None):
    """Active copy of pages to host blocks (see hs.h); int32 device tensors [n]."""
    _check("hs_active_copy", load().hs_active_copy(
        pool, req.numel(), _ptr(req), _ptr(page), _ptr(host_block), _stream(stream)))


def hs_demote_cold_pages(pool: int, req, keep_tail, freed, n_freed, stream=None):
    """Demotion of each request's pages before its tail (see hs.h). req, keep_tail,
    n_freed int32 [n]; freed int32 [n][max_pages]."""
    _check("hs_demote_cold_pages", load().hs_demote_cold_pages(
        pool, req.numel(), _ptr(req), _ptr(keep_tail), _ptr(freed), _ptr(n_freed),
        _stream(stream)))


def hs_decode_workspace_bytes(B: int, T: int, H: int, K: int) -> int:
    return load().hs_decode_workspace_bytes(B, T, H, K)


def hs_sparse_mla_decode(pool: int, q, gathered, gathered_scale, resolved, topk_idx, req_ids,
                         sm_scale: float, out, lse, workspace=None, stream=None):
    """Sparse MLA decode (see hs.h). q bf16 [B][T][H][576], out bf16 [B][T][H][512],
    lse float32 [B][T][H]; workspace uint8 tensor of hs_decode_workspace_bytes."""
    B, T, H, _ = q.shape
    K = topk_idx.shape[1]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("hs_sparse_mla_decode", load().hs_sparse_mla_decode(
        pool, B, T, H, K, _ptr(q), _ptr(gathered), _ptr(gathered_scale), _ptr(resolved),
        _ptr(topk_idx), _ptr(req_ids), float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace),
        ws, _stream(stream)))


def hs_sparse_mla_decode_per_token(pool: int, q, gathered, gathered_scale, resolved, topk_idx,
                                   req_ids, sm_scale: float, out, lse, workspace=None,
                                   stream=None):
    """Decode with one list per query token (see hs.h). q bf16 [B][T][H][576];
    topk_idx / resolved int32 [B][T][K]; gathered [B][T][K][row_bytes] or None;
    workspace of hs_decode_workspace_bytes(B*T, 1, H, K) bytes."""
    B, T, H, _ = q.shape
    K = topk_idx.shape[-1]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("hs_sparse_mla_decode_per_token", load().hs_sparse_mla_decode_per_token(
        pool, B, T, H, K, _ptr(q), _ptr(gathered), _ptr(gathered_scale), _ptr(resolved),
        _ptr(topk_idx), _ptr(req_ids), float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace),
        ws, _stream(stream)))


def hs_sparse_mla_decode_static_ws(pool: int, q, gathered, gathered_scale, resolved, topk_idx,
                                   req_ids, sm_scale: float, out, lse, stream=None):
    """hs_sparse_mla_decode without a workspace argument, for callers that cannot
    allocate device memory: the split-KV partials use a fixed array inside the
    library (HS_STATIC_DECODE_WS_BYTES; see hs.h for the sharing rules)."""
    B, T, H, _ = q.shape
    K = topk_idx.shape[1]
    _check("hs_sparse_mla_decode_static_ws", load().hs_sparse_mla_decode_static_ws(
        pool, B, T, H, K, _ptr(q), _ptr(gathered), _ptr(gathered_scale), _ptr(resolved),
        _ptr(topk_idx), _ptr(req_ids), float(sm_scale), _ptr(out), _ptr(lse), _stream(stream)))


def hs_append_rows(pool: int, rows, req_ids, start=None, index=None, stream=None):
    """New tokens' rows into the cache (see hs.h). rows bf16 [B][T][576]; req_ids
    int32 [B]; start int32 [B] or None (ctx_len - T); index int32 [B][T] or None."""
    B, T = rows.shape[0], rows.shape[1]
    _check("hs_append_rows", load().hs_append_rows(
        pool, B, T, _arg("rows", rows, "bfloat16", B, T, 576), _arg("req_ids", req_ids, "int32", B),
        _arg("start", start, "int32", B, optional=True),
        _arg("index", index, "int32", B, T, optional=True), _stream(stream)))


def _means_shape(pool: int):
    cfg = hs_pool_config()
    _check("hs_pool_get_config", load().hs_pool_get_config(pool, C.byref(cfg)))
    return cfg.max_requests, (cfg.max_ctx + 63) // 64, 576


def hs_page_means(pool: int, req, page, means, stream=None, means_shape=None):
    """Mean rows of pages (see hs.h). req, page int32 [n]; means bf16
    [max_requests][max_pages][576] (means_shape: that shape, where it is known)."""
    n = req.shape[0]
    _check("hs_page_means", load().hs_page_means(
        pool, n, _arg("req", req, "int32", n), _arg("page", page, "int32", n),
        _arg("means", means, "bfloat16", *(means_shape or _means_shape(pool))), _stream(stream)))


def hs_select_workspace_bytes(pool: int, B: int, T: int) -> int:
    return load().hs_select_workspace_bytes(pool, B, T)


def hs_select_pages(pool: int, q, means, req_ids, pages, n_first: int = 1, n_last: int = 1,
                    tree=None, topk_idx=None, workspace=None, stream=None, means_shape=None):
    """Pages of the highest score for each query token (see hs.h). q bf16
    [B][T][H][576]; means as hs_page_means; pages int32 [B][T][N] out; tree int64
    [B][T] or None; topk_idx int32 [B][T][N*64] out or None; workspace uint8 tensor
    of hs_select_workspace_bytes."""
    B, T, H = q.shape[:3]
    N = pages.shape[-1]
    ws, wp = _ws(workspace)
    _check("hs_select_pages", load().hs_select_pages(
        pool, B, T, H, N, n_first, n_last, _arg("q", q, "bfloat16", B, T, H, 576),
        _arg("means", means, "bfloat16", *(means_shape or _means_shape(pool))),
        _arg("req_ids", req_ids, "int32", B), _arg("tree", tree, "int64", B, T, optional=True),
        _arg("pages", pages, "int32", B, T, N),
        _arg("topk_idx", topk_idx, "int32", B, T, N * 64, optional=True), wp, ws, _stream(stream)))


def hs_page_decode_workspace_bytes(B: int, T: int, H: int, N: int) -> int:
    return load().hs_page_decode_workspace_bytes(B, T, H, N)


def hs_page_mla_decode(pool: int, q, pages, req_ids, tree, sm_scale: float, out, lse,
                       workspace=None, stream=None, n_pages: int = 0):
    """MLA decode over whole pages (see hs.h). q bf16 [B][T][H][576]; pages int32
    [B][N], or None for every page (planned for n_pages, 0: max_pages); tree int64
    [B][T] or None; out bf16 [B][T][H][512]; lse float32 [B][T][H]."""
    B, T, H = q.shape[:3]
    N = n_pages if pages is None else pages.shape[-1]
    ws, wp = _ws(workspace)
    _check("hs_page_mla_decode", load().hs_page_mla_decode(
        pool, B, T, H, N, _arg("q", q, "bfloat16", B, T, H, 576),
        _arg("pages", pages, "int32", B, N, optional=True), _arg("req_ids", req_ids, "int32", B),
        _arg("tree", tree, "int64", B, T, optional=True), float(sm_scale),
        _arg("out", out, "bfloat16", B, T, H, 512), _arg("lse", lse, "float32", B, T, H), wp, ws,
        _stream(stream)))


def hs_page_mla_decode_per_token(pool: int, q, pages, req_ids, tree, sm_scale: float, out, lse,
                                 workspace=None, stream=None):
    """hs_page_mla_decode with one list per query token: pages int32 [B][T][N];
    workspace of hs_page_decode_workspace_bytes(B*T, 1, H, N) bytes."""
    B, T, H = q.shape[:3]
    N = pages.shape[-1]
    ws, wp = _ws(workspace)
    _check("hs_page_mla_decode_per_token", load().hs_page_mla_decode_per_token(
        pool, B, T, H, N, _arg("q", q, "bfloat16", B, T, H, 576),
        _arg("pages", pages, "int32", B, T, N), _arg("req_ids", req_ids, "int32", B),
        _arg("tree", tree, "int64", B, T, optional=True), float(sm_scale),
        _arg("out", out, "bfloat16", B, T, H, 512), _arg("lse", lse, "float32", B, T, H), wp, ws,
        _stream(stream)))


def hs_window_workspace_bytes(pool: int, B: int, T: int, H: int, window: int, n_sink: int) -> int:
    return load().hs_window_workspace_bytes(pool, B, T, H, window, n_sink)


def hs_page_mla_decode_window(pool: int, q, req_ids, tree, window: int, n_sink: int,
                              sm_scale: float, out, lse, workspace=None, stream=None):
    """hs_page_mla_decode over the last `window` positions and the first n_sink ones (see
    hs.h); workspace of hs_window_workspace_bytes."""
    B, T, H = q.shape[:3]
    ws, wp = _ws(workspace)
    _check("hs_page_mla_decode_window", load().hs_page_mla_decode_window(
        pool, B, T, H, window, n_sink, _arg("q", q, "bfloat16", B, T, H, 576),
        _arg("req_ids", req_ids, "int32", B), _arg("tree", tree, "int64", B, T, optional=True),
        float(sm_scale), _arg("out", out, "bfloat16", B, T, H, 512),
        _arg("lse", lse, "float32", B, T, H), wp, ws, _stream(stream)))


def _table_shape(pool: int):
    return _means_shape(pool)[:2]


def hs_weights_workspace_bytes(pool: int, B: int, T: int, H: int) -> int:
    return load().hs_weights_workspace_bytes(pool, B, T, H)


def hs_page_weights(pool: int, q, lse, req_ids, tree, sm_scale: float, weights, prior=None,
                    decay: float = 1.0, workspace=None, stream=None, table_shape=None):
    """The attention weight that each page gets from the query rows q (see hs.h). q bf16
    [B][T][H][576]; lse float32 [B][T][H]; weights, prior float32 [max_requests][max_pages]
    (prior: weights itself, another tensor or None)."""
    B, T, H = q.shape[:3]
    shape = table_shape or _table_shape(pool)
    ws, wp = _ws(workspace)
    out = _arg("weights", weights, "float32", *shape)
    old = out if prior is weights else _arg("prior", prior, "float32", *shape, optional=True)
    _check("hs_page_weights", load().hs_page_weights(
        pool, B, T, H, _arg("q", q, "bfloat16", B, T, H, 576), _arg("lse", lse, "float32", B, T, H),
        _arg("req_ids", req_ids, "int32", B), _arg("tree", tree, "int64", B, T, optional=True),
        float(sm_scale), float(decay), old, out, wp, ws, _stream(stream)))


def hs_evict_pages(pool: int, req, budget, weights, kept, freed, n_freed, n_first: int = 1,
                   n_last: int = 1, saved_only: bool = False, plan: bool = False, stream=None,
                   table_shape=None):
    """Each request's pages of the least weight lose their GPU block (see hs.h). req, budget,
    n_freed int32 [n]; weights float32 [max_requests][max_pages]; kept int32 [n][N] and freed
    int32 [n][max_pages] out. plan: the lists only."""
    n, N = kept.shape
    shape = table_shape or _table_shape(pool)
    flags = (HS_EVICT_SAVED_ONLY if saved_only else 0) | (HS_EVICT_PLAN if plan else 0)
    _check("hs_evict_pages", load().hs_evict_pages(
        pool, n, N, n_first, n_last, flags, _arg("req", req, "int32", n),
        _arg("budget", budget, "int32", n), _arg("weights", weights, "float32", *shape),
        _arg("kept", kept, "int32", n, N), _arg("freed", freed, "int32", n, shape[1]),
        _arg("n_freed", n_freed, "int32", n), _stream(stream)))


_prob_dtypes: dict = {}


def _prob_rows(name: str, t, B: int, rows: int, V: int):
    """Pointer, distance of rows and hs_prob_dtype of probabilities [B][rows][V], whose rows may
    lie further apart than V values, all equally far."""
    try:  # one look, as in _arg
        if (t.shape == (B, rows, V) and t.get_device() == _only_device and t.is_contiguous()
                and B * rows > 0):
            return t.data_ptr(), V, _prob_dtypes[t.dtype]
    except (AttributeError, KeyError):
        pass
    import torch
    if not _prob_dtypes:
        _prob_dtypes.update({torch.float32: HS_PROB_F32, torch.bfloat16: HS_PROB_BF16})
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.dtype not in _prob_dtypes:
        raise ValueError(f"{name}: expected float32 or bfloat16, got {t.dtype}")
    if t.shape != (B, rows, V):
        raise ValueError(f"{name}: expected shape {[B, rows, V]}, got {list(t.shape)}")
    if t.get_device() != _only_device:
        dev = torch.cuda.current_device()
        if t.get_device() != dev:
            raise ValueError(f"{name}: on CUDA device {t.get_device()}, the current one is {dev}")
    if B * rows == 0:
        return None, V, _prob_dtypes[t.dtype]
    sb, sr, sv = t.stride()
    ld = sr if rows > 1 else (sb if B > 1 else V)
    if (V > 1 and sv != 1) or ld < V or (rows > 1 and B > 1 and sb != rows * ld):
        raise ValueError(f"{name}: expected rows of {V} contiguous values, equally far apart")
    return t.data_ptr(), ld, _prob_dtypes[t.dtype]


def hs_verify_drafts(pool: int, tokens, probs, draft_probs, tree, uniform, index, count, next_token,
                     stream=None):
    """The accepted part of each draft and the token after it (see hs.h). tokens int32 [B][T];
    probs float32 or bfloat16 [B][T][V], draft_probs the same [B][T-1][V] or None (rows of
    either may be a wider buffer's, [..., :V]); tree int64 [B][T] or None; uniform float32
    [B][T]; index int32 [B][T], count and next_token int32 [B] out."""
    B, T = tokens.shape
    V = probs.shape[-1]
    pp, ld, kind = _prob_rows("probs", probs, B, T, V)
    dp, dld = None, 0
    if draft_probs is not None:
        dp, dld, dkind = _prob_rows("draft_probs", draft_probs, B, T - 1, V)
        if dkind != kind:
            raise ValueError(f"draft_probs: expected {probs.dtype}, got {draft_probs.dtype}")
    _check("hs_verify_drafts", load().hs_verify_drafts(
        pool, B, T, V, kind, pp, ld, dp, dld, _arg("tokens", tokens, "int32", B, T),
        _arg("tree", tree, "int64", B, T, optional=True), _arg("uniform", uniform, "float32", B, T),
        _arg("index", index, "int32", B, T), _arg("count", count, "int32", B),
        _arg("next_token", next_token, "int32", B), _stream(stream)))


# ------------------------------------------------------------- convenience
class Pool:
    """Owns one hs_pool handle; methods map one-to-one onto the C ABI."""

    def __init__(self, *, dtype: int, n_gpu_blocks: int, n_host_blocks: int, max_requests: int,
                 max_ctx: int, max_topk: int, hot_rows: int = 0, stream=None):
        self.cfg = hs_pool_config(512, 64, 64, dtype, n_gpu_blocks, n_host_blocks, max_requests,
                                  max_ctx, hot_rows, max_topk)
        self.handle = hs_pool_create(self.cfg, stream)
        got = hs_pool_config()
        _check("hs_pool_get_config", load().hs_pool_get_config(self.handle, C.byref(got)))
        self.cfg = got
        t = hs_pool_tables()
        _check("hs_pool_get_tables", load().hs_pool_get_tables(self.handle, C.byref(t)))
        self._tables = t
        self.row_bytes = t.row_bytes
        self.max_pages = t.max_pages
        self.fp8 = dtype == HS_FP8_E4M3_ROWSCALE

    def close(self):
        if self.handle:
            hs_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # bookkeeping
    def request_init(self, req: int, ctx_len: int):
        _check("hs_request_init", load().hs_request_init(self.handle, req, ctx_len))

    def set_ctx_len(self, req: int, ctx_len: int):
        _check("hs_request_set_ctx_len", load().hs_request_set_ctx_len(self.handle, req, ctx_len))

    def set_ctx_lens(self, d_ctx_len, stream=None):
        """Context lengths of requests 0..n-1 from an int32 CUDA tensor."""
        _check("hs_set_ctx_len", load().hs_set_ctx_len(self.handle, _ptr(d_ctx_len),
                                                       d_ctx_len.numel(), _stream(stream)))

    def page_map(self, req: int, page: int, gpu_block: int, host_block: int):
        _check("hs_page_map", load().hs_page_map(self.handle, req, page, gpu_block, host_block))

    def page_map_range(self, req: int, first: int, gpu_blocks, host_blocks):
        g = np.ascontiguousarray(gpu_blocks, dtype=np.int32)
        h = np.ascontiguousarray(host_blocks, dtype=np.int32)
        _check("hs_page_map_range", load().hs_page_map_range(
            self.handle, req, first, len(g), g.ctypes.data, h.ctypes.data))

    def hot_lease(self, req: int, blocks):
        b = np.ascontiguousarray(blocks, dtype=np.int64)
        _check("hs_hot_lease", load().hs_hot_lease(self.handle, req, b.ctypes.data, len(b)))

    def hot_release(self, req: int):
        _check("hs_hot_release", load().hs_hot_release(self.handle, req))

    def check_bounded_wait(self, limit_us: int, stream=None):
        """Runs a device wait that nothing completes; it must time out (see hs.h)."""
        _check("hs_pool_check_bounded_wait",
               load().hs_pool_check_bounded_wait(self.handle, limit_us, _stream(stream)))

    def get_error(self) -> int:
        v = C.c_uint32()
        _check("hs_pool_get_error", load().hs_pool_get_error(self.handle, C.byref(v)))
        return v.value

    def snapshot(self) -> bytearray:
        n = C.c_size_t()
        _check("hs_pool_snapshot", load().hs_pool_snapshot(self.handle, None, 0, C.byref(n)))
        buf = bytearray(n.value)
        cbuf = (C.c_char * n.value).from_buffer(buf)
        _check("hs_pool_snapshot", load().hs_pool_snapshot(self.handle, C.addressof(cbuf),
                                                           n.value, C.byref(n)))
        return buf

    def restore(self, buf: bytearray):
        cbuf = (C.c_char * len(buf)).from_buffer(buf)
        _check("hs_pool_restore", load().hs_pool_restore(self.handle, C.addressof(cbuf), len(buf)))

    # storage views (zero-copy)
    def gpu_rows(self):
        n = self.cfg.n_gpu_blocks * 64
        return _device_view(load().hs_gpu_rows(self.handle), (n, self.row_bytes), "|u1", self)

    def gpu_scales(self):
        if not self.fp8:
            return None
        return _device_view(load().hs_gpu_scales(self.handle), (self.cfg.n_gpu_blocks * 64,), "<f4", self)

    def host_rows(self) -> np.ndarray | None:
        p = load().hs_host_rows(self.handle)
        if not p:
            return None
        n = self.cfg.n_host_blocks * 64 * self.row_bytes
        return np.ctypeslib.as_array((C.c_uint8 * n).from_address(p)).reshape(-1, self.row_bytes)

    def host_scales(self) -> np.ndarray | None:
        p = load().hs_host_scales(self.handle)
        if not p:
            return None
        n = self.cfg.n_host_blocks * 64
        return np.ctypeslib.as_array((C.c_float * n).from_address(p))

    def host_rows_device(self):
        """The host arena as seen by the GPU (reads go over the host link), or None."""
        p = load().hs_host_rows_device(self.handle)
        if not p:
            return None
        return _device_view(p, (self.cfg.n_host_blocks * 64, self.row_bytes), "|u1", self)

    def host_scales_device(self):
        p = load().hs_host_scales_device(self.handle)
        if not p:
            return None
        return _device_view(p, (self.cfg.n_host_blocks * 64,), "<f4", self)

    def tables(self) -> dict:
        t, R, C_ = self._tables, self.cfg.max_requests, self.cfg.hot_rows
        return {
            "page_table": _device_view(t.page_table, (R, self.max_pages, 2), "<i4", self),
            "hot_blocks": _device_view(t.hot_blocks, (R, C_ // 64), "<i4", self),
            "slot_tag": _device_view(t.slot_tag, (R, C_), "<i4", self),
            "slot_stamp": _device_view(t.slot_stamp, (R, C_), "<i4", self),
            "lru_order": _device_view(t.lru_order, (R, C_), "<i4", self),
            "pos_to_slot": _device_view(t.pos_to_slot, (R, self.cfg.max_ctx), "<i4", self),
            "clock": _device_view(t.clock, (R,), "<i4", self),
            "ctx_len": _device_view(t.ctx_len, (R,), "<i4", self),
        }

    # hot path
    def resolve_topk(self, req_ids, topk_idx, resolved, gathered, gathered_scale, counts,
                     stream=None):
        hs_resolve_topk(self.handle, req_ids, topk_idx, resolved, gathered, gathered_scale,
                        counts, stream)

    def sparse_mla_decode(self, q, gathered, gathered_scale, resolved, topk_idx, req_ids,
                          sm_scale, out, lse, workspace=None, stream=None):
        hs_sparse_mla_decode(self.handle, q, gathered, gathered_scale, resolved, topk_idx,
                             req_ids, sm_scale, out, lse, workspace, stream)

    def resolve_topk_union(self, req_ids, topk_idx, resolved, gathered, gathered_scale, counts,
                           stream=None):
        hs_resolve_topk_union(self.handle, req_ids, topk_idx, resolved, gathered,
                              gathered_scale, counts, stream)

    def sparse_mla_decode_per_token(self, q, gathered, gathered_scale, resolved, topk_idx,
                                    req_ids, sm_scale, out, lse, workspace=None, stream=None):
        hs_sparse_mla_decode_per_token(self.handle, q, gathered, gathered_scale, resolved,
                                       topk_idx, req_ids, sm_scale, out, lse, workspace, stream)

    # new rows, page selection, attention over pages
    def append_rows(self, rows, req_ids, start=None, index=None, stream=None):
        hs_append_rows(self.handle, rows, req_ids, start, index, stream)

    def page_means(self, req, page, means, stream=None):
        hs_page_means(self.handle, req, page, means, stream,
                      (self.cfg.max_requests, self.max_pages, 576))

    def select_pages(self, q, means, req_ids, pages, n_first=1, n_last=1, tree=None,
                     topk_idx=None, workspace=None, stream=None):
        hs_select_pages(self.handle, q, means, req_ids, pages, n_first, n_last, tree, topk_idx,
                        workspace, stream, (self.cfg.max_requests, self.max_pages, 576))

    def page_mla_decode(self, q, pages, req_ids, tree, sm_scale, out, lse, workspace=None,
                        stream=None, n_pages=0):
        hs_page_mla_decode(self.handle, q, pages, req_ids, tree, sm_scale, out, lse, workspace,
                           stream, n_pages)

    def page_mla_decode_per_token(self, q, pages, req_ids, tree, sm_scale, out, lse,
                                  workspace=None, stream=None):
        hs_page_mla_decode_per_token(self.handle, q, pages, req_ids, tree, sm_scale, out, lse,
                                     workspace, stream)

    def page_mla_decode_window(self, q, req_ids, tree, window, n_sink, sm_scale, out, lse,
                               workspace=None, stream=None):
        hs_page_mla_decode_window(self.handle, q, req_ids, tree, window, n_sink, sm_scale, out,
                                  lse, workspace, stream)

    # page weights, eviction, drafts
    def page_weights(self, q, lse, req_ids, tree, sm_scale, weights, prior=None, decay=1.0,
                     workspace=None, stream=None):
        hs_page_weights(self.handle, q, lse, req_ids, tree, sm_scale, weights, prior, decay,
                        workspace, stream, (self.cfg.max_requests, self.max_pages))

    def evict_pages(self, req, budget, weights, kept, freed, n_freed, n_first=1, n_last=1,
                    saved_only=False, plan=False, stream=None):
        hs_evict_pages(self.handle, req, budget, weights, kept, freed, n_freed, n_first, n_last,
                       saved_only, plan, stream, (self.cfg.max_requests, self.max_pages))

    def verify_drafts(self, tokens, probs, draft_probs, tree, uniform, index, count, next_token,
                      stream=None):
        hs_verify_drafts(self.handle, tokens, probs, draft_probs, tree, uniform, index, count,
                         next_token, stream)
