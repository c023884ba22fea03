"""B200 (sm_100a) paged sparse-attention prefill with page-affine query unions.

Thin Python binding over the C ABI in ``include/query_union_paged.h`` (library
``libqup.so`` built in-tree). Every step of the path runs in the library's
CUDA kernels; this module only marshals arguments. PyTorch is used for device
memory and streams. There is no CPU fallback: if the library is missing the
calls raise.

    groups = sparse_group(topk, Hq, Hkv, num_logical_pages, max_group=8, window=64)
    O = sparse_prefill_attn(Q, K_cache, V_cache, page_table, groups, q_pos, kv_len, ...)

An 8-bit cache with a scale per page and KV head, for serving: written, read (single tokens, short
runs, chunks) and evicted on the device.

    cache = KVCache(K, V, k_scale, v_scale, page_table, page_ptr, kv_len)
    cache_append(cache, k_new, v_new, tok_ptr)
    O = cache_attn(cache, Q, q_ptr, max_q, topk=None, page_weight=w)
    page_table, acc, kv_len, src = cache_evict(cache, w, acc, budget)
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import math
import os
from typing import Optional

import numpy as np

__all__ = ["Groups", "sparse_group", "sparse_prefill_attn", "build_bundles", "groups_from_host", "union_support",
           "Batch", "batch_prepare", "sparse_prefill_attn_batch", "PageItems", "page_major_items", "page_major_attn",
           "KVCache", "cache_append", "cache_attn", "cache_attn_workspace", "cache_evict", "get_error", "set_debug",
           "set_checked", "load",
           "QupError", "F32", "BF16", "E4M3", "EVICT_PAGES", "ERR"]

F32, BF16, E4M3 = 0, 1, 2
EVICT_PAGES = 24576  # QUP_CACHE_EVICT_PAGES
ERR = {"ARG": 1, "CAPACITY": 2, "CUDA": 4, "PAGE_ID": 8, "PHYS_PAGE": 16, "GROUP": 32, "TIMEOUT": 64,
       "SCALE": 128}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqup.so")
_lib = None


class QupError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {_strerror(code)} (code {code})")


_GROUP_KEYS = ("n_groups", "group_ptr", "members", "union_ptr", "union_pages", "row_mask", "counters")
_BUNDLE_KEYS = ("n_bundles", "bundle_ptr", "bundle_groups", "bunion_ptr", "bunion_pages", "bunion_mask",
                "bundle_qid", "bcounters", "bundle_order")


class _Groups(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_void_p) for k in _GROUP_KEYS] + [("cap_union", ctypes.c_int64)] +
                [(k, ctypes.c_void_p) for k in _BUNDLE_KEYS] +
                [("rows_per_group", ctypes.c_int32), ("bundle_window", ctypes.c_int32)])


class _CacheStruct(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_void_p) for k in ("K", "V", "k_scale", "v_scale", "page_table", "page_ptr", "kv_len")] +
                [(k, ctypes.c_int32) for k in ("P_phys", "Hkv", "T", "R", "total_pages", "max_pages")])


def load():
    """Load libqup.so (in-tree). Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                           "`python -m query_union_paged_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.qup_group_workspace.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(SZ), ctypes.POINTER(I64)]
    lib.qup_sparse_group.argtypes = [P, I, I, I, I, I, I, I, ctypes.POINTER(_Groups), P, SZ, P]
    lib.qup_build_bundles.argtypes = [ctypes.POINTER(_Groups), I, I, I, I, I, P, SZ, P]
    lib.qup_sparse_prefill_attn.argtypes = [P, I, P, P, I, P, P, P, I, I, I, P, I,
                                            ctypes.POINTER(_Groups), P, I, I, I, I, I,
                                            ctypes.c_float, P, P, P]
    lib.qup_get_error.argtypes = [ctypes.POINTER(I), P]
    lib.qup_error_string.argtypes = [I]
    lib.qup_error_string.restype = ctypes.c_char_p
    lib.qup_set_debug.argtypes = [I, I]
    lib.qup_num_sms.argtypes = []
    lib.qup_exp2_poly.argtypes = [P, P, I, P]
    lib.qup_union_support.argtypes = [ctypes.POINTER(_Groups), I, I, I, I, I, P, SZ, P]
    lib.qup_set_checked.argtypes = [I]
    lib.qup_batch_prepare.argtypes = [P, P, I, I, I, I, I, P, P, P, I, P, P, P, P]
    lib.qup_page_major_workspace.argtypes = [I, I, I, I, I, I, ctypes.POINTER(SZ), ctypes.POINTER(I64),
                                             ctypes.POINTER(I64), ctypes.POINTER(ctypes.c_int32)]
    lib.qup_page_major_items.argtypes = [P, I, I, I, I, I, I, ctypes.POINTER(_PageItems), P, SZ, P]
    lib.qup_page_major_attn.argtypes = [P, I, P, P, I, P, P, P, I, I, I, ctypes.POINTER(_PageItems), P, I, I, I, I,
                                        I, ctypes.c_float, P, P, P, P, P]
    lib.qup_pivot_select.argtypes = [P, P, I, P, I, I, I, I, I, I, I, I, I, I, P, P]
    lib.qup_sparse_prefill_attn_batch.argtypes = [P, I, P, P, I, P, P, P, I, I, I, P, I,
                                                  ctypes.POINTER(_Groups), P, P, I, I, I, I,
                                                  ctypes.c_float, P, P, P]
    C = ctypes.POINTER(_CacheStruct)
    lib.qup_cache_append.argtypes = [C, P, P, I, I64, I64, P, I, I, P]
    lib.qup_cache_attn_workspace.argtypes = [C, I, I, I, I, ctypes.POINTER(SZ)]
    lib.qup_cache_attn.argtypes = [C, P, I64, P, I, I, I, I, P, I, ctypes.c_float, P, P, P, P, SZ, P]
    lib.qup_cache_evict.argtypes = [C, P, P, ctypes.c_float, I, I, I, P, P, P, P, P]
    for fn in ("qup_cache_append", "qup_cache_attn_workspace", "qup_cache_attn", "qup_cache_evict",
               "qup_group_workspace", "qup_sparse_group", "qup_build_bundles", "qup_sparse_prefill_attn",
               "qup_get_error", "qup_set_debug", "qup_num_sms", "qup_exp2_poly", "qup_union_support",
               "qup_set_checked", "qup_batch_prepare", "qup_sparse_prefill_attn_batch", "qup_page_major_workspace",
               "qup_page_major_items", "qup_page_major_attn", "qup_pivot_select"):
        getattr(lib, fn).restype = I
    _lib = lib
    return lib


def _strerror(code: int) -> str:
    try:
        return load().qup_error_string(code).decode()
    except Exception:
        return str(code)


def _check(rc: int, where: str):
    if rc != 0:
        raise QupError(rc, where)


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


@dataclasses.dataclass
class Groups:
    """Device output of sparse_group (see qup_groups in the C header): the groups and the
    bundles the attention kernel walks."""
    n_groups: "torch.Tensor"
    group_ptr: "torch.Tensor"
    members: "torch.Tensor"
    union_ptr: "torch.Tensor"
    union_pages: "torch.Tensor"
    row_mask: "torch.Tensor"
    counters: "torch.Tensor"
    n_bundles: "torch.Tensor" = None
    bundle_ptr: "torch.Tensor" = None
    bundle_groups: "torch.Tensor" = None
    bunion_ptr: "torch.Tensor" = None
    bunion_pages: "torch.Tensor" = None
    bunion_mask: "torch.Tensor" = None
    bundle_qid: "torch.Tensor" = None
    bcounters: "torch.Tensor" = None
    bundle_order: "torch.Tensor" = None
    workspace: Optional["torch.Tensor"] = None
    rows_per_group: int = 0
    bundle_window: int = 0

    def c_struct(self) -> _Groups:
        cs = _Groups(*[getattr(self, k).data_ptr() for k in _GROUP_KEYS], self.union_pages.numel(),
                     *[getattr(self, k).data_ptr() for k in _BUNDLE_KEYS], self.rows_per_group,
                     self.bundle_window)
        return cs

    def _after(self, cs: _Groups):
        self.rows_per_group = cs.rows_per_group


def group_workspace(Hq, Hkv, Nq, Ksel, num_logical_pages, max_group=8, window=64):
    lib = load()
    ws = ctypes.c_size_t(0)
    cap = ctypes.c_int64(0)
    _check(lib.qup_group_workspace(Hq, Hkv, Nq, Ksel, num_logical_pages, max_group, window,
                                   ctypes.byref(ws), ctypes.byref(cap)), "qup_group_workspace")
    return ws.value, cap.value


def alloc_groups(Hq, Hkv, Nq, cap, ws_bytes, device) -> Groups:
    import torch
    i32 = dict(dtype=torch.int32, device=device)
    g = Hq // Hkv
    cap = max(int(cap), 1)
    return Groups(n_groups=torch.empty(Hkv, **i32), group_ptr=torch.empty(Hkv, Nq + 1, **i32),
                  members=torch.empty(Hkv, Nq, **i32), union_ptr=torch.empty(Hkv, Nq + 1, **i32),
                  union_pages=torch.empty(cap, **i32),
                  row_mask=torch.empty(cap, dtype=torch.int64, device=device),
                  counters=torch.empty(Hkv, 4, dtype=torch.int64, device=device),
                  n_bundles=torch.empty(Hkv, **i32), bundle_ptr=torch.empty(Hkv, Nq + 1, **i32),
                  bundle_groups=torch.empty(Hkv, Nq, **i32), bunion_ptr=torch.empty(Hkv, Nq + 1, **i32),
                  bunion_pages=torch.empty(cap, **i32), bunion_mask=torch.empty(cap, 4, **i32),
                  bundle_qid=torch.empty(Hkv, max(Nq, 1), 128 // g, **i32),
                  bcounters=torch.empty(Hkv, 2, dtype=torch.int64, device=device),
                  bundle_order=torch.empty(max(Hkv * Nq, 1), **i32),
                  workspace=torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=device))


def groups_from_host(d: dict, Hq: int, Hkv: int, num_logical_pages: int, max_group: int = 8,
                     device="cuda", stream=None) -> Groups:
    """Upload a partition held as numpy arrays (keys as the C struct: n_groups .. counters)
    and build its bundles on the device (qup_build_bundles)."""
    import torch
    Hkv_, Np1 = d["group_ptr"].shape
    Nq = Np1 - 1
    ws_bytes, cap = group_workspace(Hq, Hkv, Nq, 1, num_logical_pages, max_group, max_group)
    cap = max(cap, int(d["union_pages"].size), 1)
    gr = alloc_groups(Hq, Hkv, Nq, cap, ws_bytes, device)
    for k in _GROUP_KEYS:
        src = d[k].view("int64") if k == "row_mask" else d[k]
        dst = getattr(gr, k)
        if k in ("union_pages", "row_mask"):
            dst[:src.size].copy_(torch.from_numpy(np.ascontiguousarray(src)))
        else:
            dst.copy_(torch.from_numpy(np.ascontiguousarray(src)))
    build_bundles(gr, Hq, Hkv, Nq, num_logical_pages, max_group, stream=stream)
    return gr


def build_bundles(gr: Groups, Hq: int, Hkv: int, Nq: int, num_logical_pages: int, max_group: int = 8,
                  stream=None) -> Groups:
    lib = load()
    cs = gr.c_struct()
    _check(lib.qup_build_bundles(ctypes.byref(cs), Hq, Hkv, Nq, num_logical_pages, max_group,
                                 _p(gr.workspace), gr.workspace.numel(), _stream_ptr(stream)),
           "qup_build_bundles")
    gr._after(cs)
    return gr


def union_support(gr: Groups, Hq: int, Hkv: int, Nq: int, num_logical_pages: int, max_group: int = 8,
                  stream=None) -> Groups:
    """Every row of a group sees every page of its group's union (qup_union_support); the
    bundles are rebuilt.  Attention on the result uses the group unions as supports."""
    lib = load()
    cs = gr.c_struct()
    _check(lib.qup_union_support(ctypes.byref(cs), Hq, Hkv, Nq, num_logical_pages, max_group,
                                 _p(gr.workspace), gr.workspace.numel(), _stream_ptr(stream)),
           "qup_union_support")
    gr._after(cs)
    return gr


def sparse_group(topk, Hq: int, Hkv: int, num_logical_pages: int, max_group: int = 8,
                 window: int = 64, out: Optional[Groups] = None, stream=None,
                 bundle_window: Optional[int] = None) -> Groups:
    """Page-affinity grouping of the queries of every KV head, then bundling (qup_sparse_group).

    topk: int32 CUDA tensor [Hq][Nq][Ksel], -1 = padding. Returns Groups on the device.
    bundle_window: groups per bundling window (None keeps out's setting; 0 = library default).
    """
    lib = load()
    Hq_, Nq, Ksel = topk.shape
    assert Hq_ == Hq and topk.is_cuda and topk.is_contiguous()
    ws_bytes, cap = group_workspace(Hq, Hkv, Nq, Ksel, num_logical_pages, max_group, window)
    if out is None:
        out = alloc_groups(Hq, Hkv, Nq, cap, ws_bytes, topk.device)
    if bundle_window is not None:
        out.bundle_window = int(bundle_window)
    cs = out.c_struct()
    _check(lib.qup_sparse_group(_p(topk), Hq, Hkv, Nq, Ksel, num_logical_pages, max_group, window,
                                ctypes.byref(cs), _p(out.workspace), out.workspace.numel(),
                                _stream_ptr(stream)), "qup_sparse_group")
    out._after(cs)
    return out


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return E4M3
    raise ValueError(f"unsupported dtype {t.dtype}")


def sparse_prefill_attn(Q, K_cache, V_cache, page_table, groups: Groups, q_pos, kv_len: int,
                        k_scale=None, v_scale=None, topk=None, softmax_scale: Optional[float] = None,
                        out=None, lse=None, num_logical_pages: Optional[int] = None, stream=None):
    """Union attention over the groups (qup_sparse_prefill_attn).

    Q [Nq][Hq][d] bf16/fp32; K_cache, V_cache [P_phys][Hkv][T][d] bf16/fp32/E4M3 (uint8 or
    float8_e4m3fn, with fp32 k_scale/v_scale [Hkv]); page_table int32 [pages]; q_pos int32 [Nq].
    Returns O [Nq][Hq][d] in Q's dtype (and fills lse [Nq][Hq] fp32 if given).
    """
    import torch
    lib = load()
    Nq, Hq, d = Q.shape
    P_phys, Hkv, T, d2 = K_cache.shape
    assert d2 == d and V_cache.shape == K_cache.shape
    for t in (Q, K_cache, V_cache, page_table, q_pos):
        assert t.is_cuda and t.is_contiguous()
    if out is None:
        out = torch.empty_like(Q)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    if num_logical_pages is None:
        num_logical_pages = page_table.numel()
    cs = groups.c_struct()
    ksel = topk.shape[-1] if topk is not None else 0
    _check(lib.qup_sparse_prefill_attn(_p(Q), _dtype_code(Q), _p(K_cache), _p(V_cache),
                                       _dtype_code(K_cache), _p(k_scale), _p(v_scale), _p(page_table),
                                       num_logical_pages, P_phys, T, _p(topk), ksel, ctypes.byref(cs),
                                       _p(q_pos), kv_len, Hq, Hkv, Nq, d, float(softmax_scale),
                                       _p(out), _p(lse), _stream_ptr(stream)),
           "qup_sparse_prefill_attn")
    return out


class _PageItems(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("n_items", "item_ptr", "item_pages", "item_mask", "item_qid",
                                               "item_slot", "item_order", "row_off")] + \
               [("item_cap", ctypes.c_int64), ("slot_cap", ctypes.c_int64), ("tile_pages", ctypes.c_int32)]


@dataclasses.dataclass
class PageItems:
    """Device arrays of page-major items (see qup_page_items) and the partial-result buffers."""
    arrays: dict
    item_cap: int
    slot_cap: int
    tile_pages: int
    workspace: "torch.Tensor"
    part_o: "torch.Tensor"
    part_lse: "torch.Tensor"

    def c_struct(self) -> _PageItems:
        a = self.arrays
        return _PageItems(*[a[k].data_ptr() for k in ("n_items", "item_ptr", "item_pages", "item_mask", "item_qid",
                                                      "item_slot", "item_order", "row_off")],
                          self.item_cap, self.slot_cap, self.tile_pages)


def page_major_items(topk, Hq: int, Hkv: int, num_logical_pages: int, T: int, out: Optional[PageItems] = None,
                     stream=None) -> PageItems:
    """Page-major items of the TopK rows (qup_page_major_items): tiles of 256 tokens and the
    queries that meet them, with per-row partial slots."""
    import torch
    lib = load()
    Hq_, Nq, Ksel = topk.shape
    ws, icap, scap, tp = ctypes.c_size_t(0), ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int32(0)
    _check(lib.qup_page_major_workspace(Hq, Hkv, Nq, Ksel, num_logical_pages, T, ctypes.byref(ws), ctypes.byref(icap),
                                        ctypes.byref(scap), ctypes.byref(tp)), "qup_page_major_workspace")
    if out is None:
        dev = topk.device
        i32 = dict(dtype=torch.int32, device=dev)
        g = Hq // Hkv
        n = Hkv * icap.value
        arrays = dict(n_items=torch.empty(Hkv, **i32), item_ptr=torch.empty(Hkv, icap.value + 1, **i32),
                      item_pages=torch.empty(n * tp.value, **i32), item_mask=torch.empty(n * tp.value, 4, **i32),
                      item_qid=torch.empty(Hkv, icap.value, 128 // g, **i32), item_slot=torch.empty(n, 128, **i32),
                      item_order=torch.empty(n, **i32),
                      row_off=torch.empty(Hq * Nq + 1, dtype=torch.int64, device=dev))
        out = PageItems(arrays=arrays, item_cap=icap.value, slot_cap=scap.value, tile_pages=tp.value,
                        workspace=torch.empty(max(ws.value, 1), dtype=torch.uint8, device=dev),
                        part_o=torch.empty(scap.value, 128, dtype=torch.float32, device=dev),
                        part_lse=torch.empty(scap.value, dtype=torch.float32, device=dev))
    cs = out.c_struct()
    _check(lib.qup_page_major_items(_p(topk), Hq, Hkv, Nq, Ksel, num_logical_pages, T, ctypes.byref(cs),
                                    _p(out.workspace), out.workspace.numel(), _stream_ptr(stream)),
           "qup_page_major_items")
    out.tile_pages = cs.tile_pages
    return out


def page_major_attn(Q, K_cache, V_cache, page_table, items: PageItems, q_pos, kv_len: int, k_scale=None,
                    v_scale=None, softmax_scale: Optional[float] = None, out=None, lse=None,
                    num_logical_pages: Optional[int] = None, stream=None):
    """Page-major attention over the items (qup_page_major_attn): partial results per row and
    tile, then their merge.  Returns O [Nq][Hq][d] in Q's dtype."""
    import torch
    lib = load()
    Nq, Hq, d = Q.shape
    P_phys, Hkv, T, d2 = K_cache.shape
    if out is None:
        out = torch.empty_like(Q)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    if num_logical_pages is None:
        num_logical_pages = page_table.numel()
    cs = items.c_struct()
    _check(lib.qup_page_major_attn(_p(Q), _dtype_code(Q), _p(K_cache), _p(V_cache), _dtype_code(K_cache),
                                   _p(k_scale), _p(v_scale), _p(page_table), num_logical_pages, P_phys, T,
                                   ctypes.byref(cs), _p(q_pos), kv_len, Hq, Hkv, Nq, d, float(softmax_scale),
                                   _p(items.part_o), _p(items.part_lse), _p(out), _p(lse), _stream_ptr(stream)),
           "qup_page_major_attn")
    return out


@dataclasses.dataclass
class Batch:
    """Device arrays of batched requests after batch_prepare (see qup_batch_prepare)."""
    q_ptr: "torch.Tensor"
    page_ptr: "torch.Tensor"
    kv_len: "torch.Tensor"
    topk_global: "torch.Tensor"
    q_end: "torch.Tensor"
    page_len: "torch.Tensor"
    total_pages: int


def batch_prepare(topk, q_pos, q_ptr, page_ptr, kv_len, total_pages: int, T: int, stream=None) -> Batch:
    """Rebase request-local TopK rows and positions to the concatenated page space of a batch
    (qup_batch_prepare).  topk int32 [Hq][Nq][Ksel], q_pos int32 [Nq]; q_ptr, page_ptr int32 [R+1];
    kv_len int32 [R]; all CUDA tensors."""
    import torch
    Hq, Nq, Ksel = topk.shape
    R = q_ptr.numel() - 1
    dev = topk.device
    b = Batch(q_ptr=q_ptr, page_ptr=page_ptr, kv_len=kv_len,
              topk_global=torch.empty_like(topk), q_end=torch.empty(Nq, dtype=torch.int32, device=dev),
              page_len=torch.empty(max(total_pages, 1), dtype=torch.int32, device=dev), total_pages=total_pages)
    _check(load().qup_batch_prepare(_p(topk), _p(q_pos), Hq, Nq, Ksel, T, R, _p(q_ptr), _p(page_ptr), _p(kv_len),
                                    total_pages, _p(b.topk_global), _p(b.q_end), _p(b.page_len),
                                    _stream_ptr(stream)), "qup_batch_prepare")
    return b


def pivot_select(q_idx, page_key, q_pos, g: int, T: int, group_size: int, n_cand: int, K: int,
                 refine: bool = True, out=None, stream=None):
    """Proxy-query page selection (qup_pivot_select): TopK page IDs per (query head, query) for
    sparse_group.  q_idx [Nq][Hkv][d_idx] and page_key [P][Hkv][d_idx] bf16 or fp32 CUDA tensors,
    q_pos int32 [Nq]; returns int32 [Hkv*g][Nq][K] (-1 padded)."""
    import torch
    Nq, Hkv, d = q_idx.shape
    P = page_key.shape[0]
    assert page_key.shape[1:] == (Hkv, d) and page_key.dtype == q_idx.dtype
    if out is None:
        out = torch.empty((Hkv * g, Nq, K), dtype=torch.int32, device=q_idx.device)
    _check(load().qup_pivot_select(_p(q_idx), _p(page_key), _dtype_code(q_idx), _p(q_pos), Nq, Hkv, g, d, P, T,
                                   group_size, n_cand, K, 1 if refine else 0, _p(out), _stream_ptr(stream)),
           "qup_pivot_select")
    return out


def sparse_prefill_attn_batch(Q, K_cache, V_cache, page_table, groups: Groups, batch: Batch, k_scale=None,
                              v_scale=None, softmax_scale: Optional[float] = None, out=None, lse=None,
                              checked_topk: bool = False, stream=None):
    """Union attention over batched requests (qup_sparse_prefill_attn_batch): page_table is the
    concatenated table of batch.total_pages entries; groups come from sparse_group on
    batch.topk_global."""
    import torch
    lib = load()
    Nq, Hq, d = Q.shape
    P_phys, Hkv, T, d2 = K_cache.shape
    assert d2 == d and V_cache.shape == K_cache.shape
    if out is None:
        out = torch.empty_like(Q)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    cs = groups.c_struct()
    tk = batch.topk_global if checked_topk else None
    _check(lib.qup_sparse_prefill_attn_batch(_p(Q), _dtype_code(Q), _p(K_cache), _p(V_cache), _dtype_code(K_cache),
                                             _p(k_scale), _p(v_scale), _p(page_table), batch.total_pages, P_phys, T,
                                             _p(tk), tk.shape[-1] if tk is not None else 0, ctypes.byref(cs),
                                             _p(batch.q_end), _p(batch.page_len), Hq, Hkv, Nq, d,
                                             float(softmax_scale), _p(out), _p(lse), _stream_ptr(stream)),
           "qup_sparse_prefill_attn_batch")
    return out


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


_2_31 = 1 << 31


def _int32(**numbers):
    """The numbers fit the C call's int (ctypes would cut them without a word)."""
    for name, x in numbers.items():
        _need(-_2_31 <= x < _2_31, f"{name} {x}: out of 32 bits")


def _whole(t, name: str, dtype, shape, index: int):
    """t is a contiguous tensor of this type and shape on device `index`.  The message is put together only
    when it is needed: these checks are most of what a short call costs on the host."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
        return
    raise ValueError(f"{name}: contiguous {dtype} {tuple(shape)} on device {index} wanted, got {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _heads(t, name: str, dtype, shape, index: int):
    """As _whole, but with any stride between the rows of the first dimension."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == index and
            (t.is_contiguous() or (t.stride(2) == 1 and t.stride(1) == 128))):
        return
    raise ValueError(f"{name}: {dtype} {tuple(shape)} with contiguous heads on device {index} wanted, got {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


class KVCache:
    """An 8-bit KV cache of R requests with one scale per (page, KV head): qup_cache in the C header.

    K, V [P_phys][Hkv][T][128] uint8 or float8_e4m3fn; k_scale, v_scale fp32 [P_phys][Hkv];
    page_table int32 [total_pages], request r's logical pages being the entries
    page_ptr[r] .. page_ptr[r+1); page_ptr int32 [R+1]; kv_len int32 [R], the tokens of each request.
    max_pages: page table entries of one request, at most (default: all of them, and for cache_evict
    EVICT_PAGES pages with tokens, if that is less).

    The object keeps the tensors and passes their addresses: their contents may change (kv_len grows,
    the page table is rewritten by cache_evict), the tensors may not be replaced.
    """

    __slots__ = ("K", "V", "k_scale", "v_scale", "page_table", "page_ptr", "kv_len", "max_pages", "device", "R", "Hkv",
                 "total_pages", "_c", "_ref", "_evict_c", "_evict_ref", "_index")

    def __init__(self, K, V, k_scale, v_scale, page_table, page_ptr, kv_len, max_pages: Optional[int] = None):
        import torch
        _need(K.dim() == 4 and K.shape[3] == 128, f"K: [P_phys][Hkv][T][128] wanted, got {tuple(K.shape)}")
        P_phys, Hkv, T, _ = K.shape
        index = K.get_device()
        _need(K.dtype in (torch.uint8, torch.float8_e4m3fn), f"K: uint8 or float8_e4m3fn wanted, got {K.dtype}")
        for t, name in ((K, "K"), (V, "V")):
            _whole(t, name, K.dtype, K.shape, index)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _whole(t, name, torch.float32, (P_phys, Hkv), index)
        for t, name in ((page_table, "page_table"), (page_ptr, "page_ptr"), (kv_len, "kv_len")):
            _whole(t, name, torch.int32, (t.numel(),), index)
        _need(page_ptr.numel() == kv_len.numel() + 1, "page_ptr has one entry more than kv_len")
        _need(T in (16, 32, 64, 128), f"page size {T}: 16, 32, 64 or 128 wanted")
        _need(page_table.numel() > 0 and P_phys > 0, "an empty page table or cache")
        given = max_pages is not None
        if not given:
            max_pages = page_table.numel()
        _need(1 <= max_pages <= page_table.numel(), f"max_pages {max_pages}: 1 .. {page_table.numel()} wanted")
        _need(K.is_cuda, f"the cache is on {K.device}: CUDA tensors wanted")
        self.K, self.V, self.k_scale, self.v_scale = K, V, k_scale, v_scale
        self.page_table, self.page_ptr, self.kv_len = page_table, page_ptr, kv_len
        self.max_pages, self.device, self._index = max_pages, K.device, index
        self.R, self.Hkv, self.total_pages = kv_len.numel(), Hkv, page_table.numel()
        self._c = _CacheStruct(*[t.data_ptr() for t in (K, V, k_scale, v_scale, page_table, page_ptr, kv_len)],
                               P_phys, Hkv, T, self.R, self.total_pages, max_pages)
        self._ref = self._evict_ref = ctypes.byref(self._c)
        if not given and max_pages > EVICT_PAGES:  # no limit was given: eviction's own
            self._evict_c = _CacheStruct.from_buffer_copy(self._c)
            self._evict_c.max_pages = EVICT_PAGES
            self._evict_ref = ctypes.byref(self._evict_c)


def _made_on(stream):
    """Buffers made inside belong to the call's stream: torch's allocator then hands their memory out again in
    that stream's order, and not to the current stream while the call is still queued on the other one."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _launch(fn, where: str, index: int, stream, *args):
    """fn(*args, stream) with the cache's device current; stream: a torch stream, or None for that device's
    current one."""
    import torch
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        _need(stream.device.index == index, f"the stream is on {stream.device}, the cache on device {index}")
        raw = stream.cuda_stream
    if torch.cuda.current_device() == index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != 0:
        raise QupError(rc, where)


def cache_append(cache: KVCache, k_new, v_new, tok_ptr, stream=None):
    """Write new tokens into the cache (qup_cache_append).

    k_new, v_new [N][Hkv][128] bf16 or fp32 (a token's heads contiguous, any token stride that keeps 16-byte
    rows); tok_ptr int32 [R+1]: rows tok_ptr[r] .. tok_ptr[r+1) are request r's last tokens, which
    cache.kv_len counts already.  A page's scale grows when a new token needs it (its older tokens are
    requantised).
    """
    import torch
    index, hkv, dtype = cache._index, cache.Hkv, k_new.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"k_new: bfloat16 or float32 wanted, got {dtype}")
    N = k_new.shape[0]
    _heads(k_new, "k_new", dtype, (N, hkv, 128), index)
    _heads(v_new, "v_new", dtype, (N, hkv, 128), index)
    _whole(tok_ptr, "tok_ptr", torch.int32, (cache.R + 1,), index)
    ks, vs = (k_new.stride(0), v_new.stride(0)) if N > 1 else (hkv * 128, hkv * 128)
    _launch((_lib or load()).qup_cache_append, "qup_cache_append", index, stream, cache._ref, k_new.data_ptr(),
            v_new.data_ptr(), BF16 if dtype is torch.bfloat16 else F32, ks, vs, tok_ptr.data_ptr(), N, 128)


def cache_attn_workspace(cache: KVCache, Nq: int, Hq: int, max_q: int, page_weight: bool = False, topk: bool = True):
    """A workspace for cache_attn calls of these sizes on this cache (qup_cache_attn_workspace).  Calls that
    may run at the same time, captured graphs among them, need one each.  With page_weight, topk=False makes one
    for calls without topk only: up to T / 16 times smaller where requests are long.
    """
    import torch
    _int32(Nq=Nq, Hq=Hq, max_q=max_q)
    n = ctypes.c_size_t(0)
    _check(load().qup_cache_attn_workspace(cache._ref, Nq, max_q, Hq, (1 if topk else 2) if page_weight else 0,
                                           ctypes.byref(n)), "qup_cache_attn_workspace")
    return torch.empty(n.value, dtype=torch.uint8, device=cache.device)


def cache_attn(cache: KVCache, Q, q_ptr, max_q: int, topk=None, softmax_scale: Optional[float] = None, out=None,
               lse=None, page_weight=None, workspace=None, stream=None):
    """Attention over the cache (qup_cache_attn): decode, short runs and chunks of queries.

    Q [Nq][Hq][128] bf16 (a query's heads contiguous); q_ptr int32 [R+1]: rows q_ptr[r] .. q_ptr[r+1) are
    request r's last positions, at most max_q of them; topk int32 [Hq][Nq][Ksel] logical pages of the query's
    request (-1 = padding) or None for all pages.  Fills lse fp32 [Nq][Hq] and page_weight fp32
    [total_pages][Hkv] if given.  Returns O [Nq][Hq][128] bf16.  An output or workspace that is not given is
    made on `stream`.
    """
    import torch
    index = cache._index
    _need(Q.dim() == 3, "Q: [Nq][Hq][128] wanted")
    Nq, Hq, _ = shape = Q.shape
    if not -_2_31 <= max_q < _2_31:
        _int32(max_q=max_q)
    _heads(Q, "Q", torch.bfloat16, (Nq, Hq, 128), index)
    _whole(q_ptr, "q_ptr", torch.int32, (cache.R + 1,), index)
    ksel = topk_p = lse_p = weight_p = None
    if topk is not None:
        ksel = topk.shape[-1]
        _whole(topk, "topk", torch.int32, (Hq, Nq, ksel), index)
        topk_p = topk.data_ptr() or q_ptr.data_ptr()  # no entries: any address says that it is a TopK call
    if out is None:
        with _made_on(stream):
            out = torch.empty(shape, dtype=torch.bfloat16, device=Q.device)
    else:
        _whole(out, "out", torch.bfloat16, shape, index)
    if lse is not None:
        _whole(lse, "lse", torch.float32, (Nq, Hq), index)
        lse_p = lse.data_ptr()
    if page_weight is not None:
        _whole(page_weight, "page_weight", torch.float32, (cache.total_pages, cache.Hkv), index)
        weight_p = page_weight.data_ptr()
    if workspace is None:
        with _made_on(stream):
            workspace = cache_attn_workspace(cache, Nq, Hq, max_q, page_weight is not None, topk is not None)
    size = workspace.numel()
    _whole(workspace, "workspace", torch.uint8, (size,), index)
    _launch((_lib or load()).qup_cache_attn, "qup_cache_attn", index, stream, cache._ref, Q.data_ptr(),
            Q.stride(0) if Nq > 1 else Hq * 128, q_ptr.data_ptr(), Nq, max_q, Hq, 128, topk_p, ksel or 0,
            1.0 / math.sqrt(128) if softmax_scale is None else softmax_scale, out.data_ptr(), lse_p, weight_p,
            workspace.data_ptr(), size)
    return out


def cache_evict(cache: KVCache, page_weight, acc, budget: int, sink: int = 1, recent: int = 1, decay: float = 1.0,
                out=None, stream=None):
    """Evict whole pages by accumulated attention weight (qup_cache_evict).

    page_weight fp32 [total_pages][Hkv] of the last cache_attn, acc fp32 [total_pages]: what each page has
    gathered before.  A request with more than `budget` pages drops the lowest of decay * acc + sum of
    page_weight, but none of its first `sink` and last `recent`.  Returns (page_table, acc, kv_len, page_src),
    the compacted table, accumulator and lengths and each entry's old place in its request; `out` holds these
    four tensors if given, which may be the cache's own page_table and kv_len, and acc; else they are made on
    `stream`.
    """
    import torch
    index, n = cache._index, cache.total_pages
    if not (-_2_31 <= budget < _2_31 and -_2_31 <= sink < _2_31 and -_2_31 <= recent < _2_31):
        _int32(budget=budget, sink=sink, recent=recent)
    _whole(page_weight, "page_weight", torch.float32, (n, cache.Hkv), index)
    _whole(acc, "acc", torch.float32, (n,), index)
    if out is None:
        with _made_on(stream):
            out = (torch.empty_like(cache.page_table), torch.empty_like(acc), torch.empty_like(cache.kv_len),
                   torch.empty_like(cache.page_table))
    table, acc_out, lens, src = out
    _whole(table, "out page_table", torch.int32, (n,), index)
    _whole(acc_out, "out acc", torch.float32, (n,), index)
    _whole(lens, "out kv_len", torch.int32, (cache.R,), index)
    _whole(src, "out page_src", torch.int32, (n,), index)
    _launch((_lib or load()).qup_cache_evict, "qup_cache_evict", index, stream, cache._evict_ref, page_weight.data_ptr(),
            acc.data_ptr(), decay, budget, sink, recent, table.data_ptr(), acc_out.data_ptr(), lens.data_ptr(),
            src.data_ptr())
    return table, acc_out, lens, src


def exp2_poly(x, out=None, stream=None):
    """2^x by the attention softmax's polynomial exponential (test hook, qup_exp2_poly).
    x: float32 CUDA tensor; returns a tensor of the same shape."""
    import torch
    assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()
    if out is None:
        out = torch.empty_like(x)
    _check(load().qup_exp2_poly(_p(x), _p(out), x.numel(), _stream_ptr(stream)), "qup_exp2_poly")
    return out


def get_error(stream=None) -> int:
    """Synchronize the stream, then read and clear the device error word."""
    lib = load()
    code = ctypes.c_int(0)
    _check(lib.qup_get_error(ctypes.byref(code), _stream_ptr(stream)), "qup_get_error")
    return code.value


def set_debug(wait_limit_ms: int = 0, skip_stage: int = -1):
    _check(load().qup_set_debug(wait_limit_ms, skip_stage), "qup_set_debug")


def set_checked(on: bool):
    """Checked mode (qup_set_checked): attention calls given topk first verify every bundle row's
    page mask against its TopK row and raise the GROUP error bit on a mismatch."""
    _check(load().qup_set_checked(1 if on else 0), "qup_set_checked")


def num_sms() -> int:
    return load().qup_num_sms()
