"""ctypes binding of liblora (include/lora.h): argument marshalling only.

Every function has the name of the C entry point it calls and takes torch
tensors (device memory) or plain Python numbers; it passes their pointers
and sizes through and raises LoraError on a negative return code.  There is
no fallback: if liblora.so is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblora.so")

LORA_OK = 0
ERR_NAMES = {
    -1: "LORA_ERR_INVALID_ARG", -2: "LORA_ERR_BAD_RANK", -3: "LORA_ERR_WIDTH_MISMATCH",
    -4: "LORA_ERR_POOL_OOM", -5: "LORA_ERR_BAD_SLOT", -6: "LORA_ERR_CUDA", -7: "LORA_ERR_WORKSPACE",
    -8: "LORA_ERR_TOO_LARGE", -9: "LORA_ERR_ALL_PINNED",
}
DEV_ERR_BAD_ID = 1
DEV_ERR_EMPTY_SLOT = 2
DEV_ERR_TIMEOUT = 4
DEV_ERR_BAD_PAGE = 8
DEV_ERR_NO_PAGES = 16
DEV_ERR_BAD_LENGTH = 32
PAGE_ROWS = 16
MAX_RANK = 64
MAX_PAGES_PER_MATRIX = 4
MAX_SLOTS = 4096
OPT_LONG_SEGMENT = 1
OPT_DECODE_JOB_TOKENS = 2
OPT_GATHER_PATH = 3
GATHER_AUTO, GATHER_CLUSTER, GATHER_SPLIT = 0, 1, 2
OPT_PLAN_KERNEL = 4
PLAN_AUTO, PLAN_GENERAL = 0, 1
NOALLOC_MAX_TOKENS = 32768
NOALLOC_SCRATCH_BYTES = 2162688
MAX_JOB_TOKENS = 16
MAX_PROJECTIONS = 8
KV_GRANULE = 16
KV_GROUP = 64
KV_MAX_REQUESTS = 4096
KV_MAX_GROUP = 64
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

EXPORTS = [
    "lora_pool_create", "lora_pool_destroy", "lora_pool_free_pages", "lora_pool_num_pages",
    "lora_pool_alloc_pages", "lora_pool_free_page_list", "lora_pool_usage",
    "lora_pool_load", "lora_pool_evict", "lora_pool_read_row", "lora_workspace_size",
    "lora_plan", "lora_shrink", "lora_expand_add", "lora_expand_add_strided", "lora_apply", "lora_apply_planned", "lora_apply_noalloc",
    "lora_apply_multi", "lora_apply_multi_planned",
    "lora_slot_cache_create", "lora_slot_cache_destroy", "lora_slot_cache_acquire", "lora_slot_cache_unpin",
    "lora_slot_cache_invalidate", "lora_slot_cache_lookup", "lora_slot_cache_stats",
    "lora_kv_block_bytes", "lora_kv_layout", "lora_rope", "lora_kv_append", "lora_kv_gather",
    "lora_kv_attend_workspace_size", "lora_kv_attend", "lora_prompt_attend",
    "lora_set_option", "lora_get_option", "lora_last_cuda_error", "lora_last_launch_count",
]


class LoraProjection(ctypes.Structure):
    """lora_projection_t: one projection of lora_apply_multi."""
    _fields_ = [("Y", ctypes.c_void_p), ("d_out", ctypes.c_int), ("ranks", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("pa", ctypes.c_void_p),
                ("pb", ctypes.c_void_p)]


class LoraRows(ctypes.Structure):
    """lora_rows_t: a [T, heads, head_dim] tensor with its strides."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class LoraKvCache(ctypes.Structure):
    """lora_kv_cache_t: the pages of one layer's cache."""
    _fields_ = [("pages", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t), ("num_pages", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("block_tokens", ctypes.c_int)]


class LoraError(RuntimeError):
    def __init__(self, name: str, rc: int, detail: str = ""):
        self.rc = rc
        super().__init__(f"{name} failed: {ERR_NAMES.get(rc, rc)}{(' (' + detail + ')') if detail else ''}")


_lib = None
V = ctypes.c_void_p
I = ctypes.c_int
F = ctypes.c_float
Z = ctypes.c_size_t


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblora.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"liblora.so not found at {path}; run heterogeneous_adapter_batching_b200.build.build()")
    lib = ctypes.CDLL(path)
    sig = {
        "lora_pool_create": (I, [V, Z, I, I, ctypes.POINTER(V)]),
        "lora_pool_destroy": (I, [V]),
        "lora_pool_free_pages": (I, [V]),
        "lora_pool_num_pages": (I, [V]),
        "lora_pool_alloc_pages": (I, [V, I, V]),
        "lora_pool_free_page_list": (I, [V, V, I]),
        "lora_pool_usage": (I, [V, ctypes.POINTER(I), ctypes.POINTER(I)]),
        "lora_pool_load": (I, [V, V, I, I, I, F, V, V, V, V, V, V, V]),
        "lora_pool_evict": (I, [V, V, I, I, V, V, V, V]),
        "lora_pool_read_row": (I, [V, V, I, I, I, I, V, V]),
        "lora_workspace_size": (Z, [I, I]),
        "lora_plan": (I, [V, I, V, I, V, V, V, Z, V, V]),
        "lora_shrink": (I, [V, I, I, V, I, V, V, V, V, V, Z, V, V]),
        "lora_expand_add": (I, [V, V, I, I, V, I, V, V, V, V, V, Z, V, V]),
        "lora_expand_add_strided": (I, [V, V, I, I, I, V, I, V, V, V, V, V, Z, V, V]),
        "lora_apply": (I, [V, V, I, I, I, V, I, V, V, V, V, V, V, Z, V, V]),
        "lora_apply_planned": (I, [V, V, I, I, I, I, V, V, V, V, V, V, Z, V, V]),
        "lora_apply_noalloc": (I, [V, V, I, I, I, V, I, V, V, V, V, V, V, V]),
        "lora_apply_multi": (I, [V, I, I, V, I, ctypes.POINTER(LoraProjection), I, V, Z, V, V]),
        "lora_apply_multi_planned": (I, [V, I, I, I, ctypes.POINTER(LoraProjection), I, V, Z, V, V]),
        "lora_slot_cache_create": (I, [I, ctypes.POINTER(V)]),
        "lora_slot_cache_destroy": (I, [V]),
        "lora_slot_cache_acquire": (I, [V, ctypes.c_int64, I, ctypes.POINTER(I), ctypes.POINTER(I),
                                        ctypes.POINTER(ctypes.c_int64)]),
        "lora_slot_cache_unpin": (I, [V, I]),
        "lora_slot_cache_invalidate": (I, [V, I]),
        "lora_slot_cache_lookup": (I, [V, ctypes.c_int64, ctypes.POINTER(I)]),
        "lora_slot_cache_stats": (I, [V, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                                      ctypes.POINTER(ctypes.c_int64)]),
        "lora_kv_block_bytes": (Z, [I, I, I]),
        "lora_kv_layout": (I, [V, V, V, I, I, I, V, I, V, I, V, V, V, V, V, V, V, V, V]),
        "lora_rope": (I, [V, I, V, I, I, I, I, V, V, I, I, ctypes.c_double, V, V, I, V]),
        "lora_kv_append": (I, [V, I, V, V, I, I, V, V, I, I, ctypes.c_double, V, V, V, V, V, I, V, V]),
        "lora_kv_gather": (I, [V, V, I, V, V, I, V, V]),
        "lora_kv_attend_workspace_size": (Z, [I, I, I, I]),
        "lora_kv_attend": (I, [V, I, I, I, V, V, I, V, V, I, I, F, V, V, V, Z, V, V]),
        "lora_prompt_attend": (I, [V, V, V, I, I, I, I, I, I, V, V, I, F, V, V, V, V]),
        "lora_set_option": (I, [I, I]),
        "lora_get_option": (I, [I]),
        "lora_last_cuda_error": (ctypes.c_char_p, []),
        "lora_last_launch_count": (I, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _s(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(name: str, rc: int):
    if rc != LORA_OK:
        detail = lora_last_cuda_error() if rc == -6 else ""
        raise LoraError(name, rc, detail)
    return rc


class Pool:
    """Host handle of one page pool over a caller-owned device buffer."""

    def __init__(self, handle: int, buf: torch.Tensor, width: int):
        self.handle = handle
        self.buf = buf          # keeps the device memory alive
        self.width = width

    def __del__(self):
        try:
            if self.handle and _lib is not None:
                _lib.lora_pool_destroy(ctypes.c_void_p(self.handle))
                self.handle = 0
        except Exception:
            pass

    @property
    def _h(self):
        return ctypes.c_void_p(self.handle)


def lora_pool_create(dev_buf: torch.Tensor, width: int, page_rows: int = PAGE_ROWS) -> Pool:
    lib = load_library()
    out = ctypes.c_void_p()
    nbytes = dev_buf.numel() * dev_buf.element_size()
    _check("lora_pool_create", lib.lora_pool_create(_p(dev_buf), nbytes, width, page_rows, ctypes.byref(out)))
    return Pool(out.value, dev_buf, width)


def lora_pool_destroy(pool: Pool) -> None:
    if pool.handle:
        load_library().lora_pool_destroy(pool._h)
        pool.handle = 0


def lora_pool_free_pages(pool: Pool) -> int:
    return load_library().lora_pool_free_pages(pool._h)


def lora_pool_num_pages(pool: Pool) -> int:
    return load_library().lora_pool_num_pages(pool._h)


def lora_pool_alloc_pages(pool: Pool, n: int) -> torch.Tensor:
    """n free pages of the pool for another tenant (KV blocks); host int32 ids."""
    ids = torch.empty(max(n, 0), dtype=torch.int32)
    _check("lora_pool_alloc_pages", load_library().lora_pool_alloc_pages(pool._h, n, _p(ids) if n > 0 else None))
    return ids


def lora_pool_free_page_list(pool: Pool, ids: torch.Tensor) -> None:
    ids = ids.to(torch.int32).contiguous()
    assert ids.device.type == "cpu"
    _check("lora_pool_free_page_list", load_library().lora_pool_free_page_list(
        pool._h, _p(ids) if ids.numel() else None, ids.numel()))


def lora_pool_usage(pool: Pool):
    """(pages held by adapters, pages held through lora_pool_alloc_pages)."""
    a, o = ctypes.c_int(), ctypes.c_int()
    _check("lora_pool_usage", load_library().lora_pool_usage(pool._h, ctypes.byref(a), ctypes.byref(o)))
    return a.value, o.value


def lora_pool_load(pa: Pool, pb: Pool, slot: int, num_slots: int, rank: int, alpha: float,
                   a_t: torch.Tensor, b: torch.Tensor, page_ids: Optional[torch.Tensor],
                   page_table: torch.Tensor, scales: torch.Tensor, ranks: torch.Tensor, stream=None) -> None:
    """a_t: [rank, d_in] bf16 (host or device), b: [rank, d_out] bf16; page_ids: host int32 [2, 4] or None."""
    if page_ids is not None:
        assert page_ids.device.type == "cpu" and page_ids.dtype == torch.int32 and page_ids.is_contiguous()
    _check("lora_pool_load", load_library().lora_pool_load(
        pa._h, pb._h, slot, num_slots, rank, alpha, _p(a_t), _p(b), _p(page_ids),
        _p(page_table), _p(scales), _p(ranks), _s(stream)))


def lora_pool_evict(pa: Pool, pb: Pool, slot: int, num_slots: int, page_table: torch.Tensor,
                    scales: torch.Tensor, ranks: torch.Tensor, stream=None) -> None:
    _check("lora_pool_evict", load_library().lora_pool_evict(
        pa._h, pb._h, slot, num_slots, _p(page_table), _p(scales), _p(ranks), _s(stream)))


def lora_pool_read_row(pool: Pool, page_table: torch.Tensor, num_slots: int, slot: int, m: int, k: int,
                       out: torch.Tensor, stream=None) -> None:
    _check("lora_pool_read_row", load_library().lora_pool_read_row(
        pool._h, _p(page_table), num_slots, slot, m, k, _p(out), _s(stream)))


def lora_workspace_size(T: int, num_slots: int) -> int:
    return int(load_library().lora_workspace_size(T, num_slots))


def lora_plan(ids, T, ranks, num_slots, perm_out, seg_start_out, ws, err=None, stream=None) -> None:
    _check("lora_plan", load_library().lora_plan(
        _p(ids), T, _p(ranks), num_slots, _p(perm_out), _p(seg_start_out), _p(ws),
        ws.numel() * ws.element_size(), _p(err), _s(stream)))


def lora_shrink(X, T, d_in, ids, num_slots, ranks, page_table, pa: Pool, V, ws, err=None, stream=None) -> None:
    _check("lora_shrink", load_library().lora_shrink(
        _p(X), T, d_in, _p(ids), num_slots, _p(ranks), _p(page_table), pa._h, _p(V), _p(ws),
        ws.numel() * ws.element_size(), _p(err), _s(stream)))


def lora_expand_add(V, Y, T, d_out, ids, num_slots, ranks, scales, page_table, pb: Pool, ws, err=None,
                    stream=None) -> None:
    _check("lora_expand_add", load_library().lora_expand_add(
        _p(V), _p(Y), T, d_out, _p(ids), num_slots, _p(ranks), _p(scales), _p(page_table), pb._h, _p(ws),
        ws.numel() * ws.element_size(), _p(err), _s(stream)))


def lora_expand_add_strided(V, Y, ldy, T, d_out, ids, num_slots, ranks, scales, page_table, pb: Pool, ws, err=None,
                            stream=None) -> None:
    """Y: a [T, d_out] column block of a wider fp32 tensor whose rows are ldy apart."""
    _check("lora_expand_add_strided", load_library().lora_expand_add_strided(
        _p(V), _p(Y), ldy, T, d_out, _p(ids), num_slots, _p(ranks), _p(scales), _p(page_table), pb._h, _p(ws),
        ws.numel() * ws.element_size(), _p(err), _s(stream)))


def lora_apply(X, Y, T, d_in, d_out, ids, num_slots, ranks, scales, page_table, pa: Pool, pb: Pool, ws,
               err=None, stream=None) -> None:
    _check("lora_apply", load_library().lora_apply(
        _p(X), _p(Y), T, d_in, d_out, _p(ids), num_slots, _p(ranks), _p(scales), _p(page_table),
        pa._h, pb._h, _p(ws), ws.numel() * ws.element_size(), _p(err), _s(stream)))


def lora_apply_planned(X, Y, T, d_in, d_out, num_slots, ranks, scales, page_table, pa: Pool, pb: Pool, ws,
                       err=None, stream=None) -> None:
    _check("lora_apply_planned", load_library().lora_apply_planned(
        _p(X), _p(Y), T, d_in, d_out, num_slots, _p(ranks), _p(scales), _p(page_table),
        pa._h, pb._h, _p(ws), ws.numel() * ws.element_size(), _p(err), _s(stream)))


def lora_apply_noalloc(X, Y, T, d_in, d_out, ids, num_slots, ranks, scales, page_table, pa: Pool, pb: Pool,
                       err=None, stream=None) -> None:
    """lora_apply without a workspace: the plan lives in the library's fixed device
    scratch, for callers that cannot allocate device memory (see include/lora.h)."""
    _check("lora_apply_noalloc", load_library().lora_apply_noalloc(
        _p(X), _p(Y), T, d_in, d_out, _p(ids), num_slots, _p(ranks), _p(scales), _p(page_table),
        pa._h, pb._h, _p(err), _s(stream)))


def _proj_array(projs):
    arr = (LoraProjection * len(projs))()
    for i, (Y, d_out, ranks, scales, page_table, pa, pb) in enumerate(projs):
        arr[i] = LoraProjection(Y.data_ptr(), d_out, ranks.data_ptr(), scales.data_ptr(), page_table.data_ptr(),
                                pa.handle, pb.handle)
    return arr


def lora_apply_multi(X, T, d_in, ids, num_slots, projs, ws, err=None, stream=None) -> None:
    """projs: sequence of (Y, d_out, ranks, scales, page_table, pa: Pool, pb: Pool)."""
    _check("lora_apply_multi", load_library().lora_apply_multi(
        _p(X), T, d_in, _p(ids), num_slots, _proj_array(projs), len(projs), _p(ws), ws.numel() * ws.element_size(),
        _p(err), _s(stream)))


def lora_apply_multi_planned(X, T, d_in, num_slots, projs, ws, err=None, stream=None) -> None:
    _check("lora_apply_multi_planned", load_library().lora_apply_multi_planned(
        _p(X), T, d_in, num_slots, _proj_array(projs), len(projs), _p(ws), ws.numel() * ws.element_size(),
        _p(err), _s(stream)))


class SlotCache:
    """lora_slot_cache_t: which adapter key lives in which slot (exact LRU over
    the slots no running batch pins).  Host bookkeeping only."""

    def __init__(self, num_slots: int):
        h = ctypes.c_void_p()
        _check("lora_slot_cache_create", load_library().lora_slot_cache_create(num_slots, ctypes.byref(h)))
        self.handle = h.value
        self.num_slots = num_slots
        self._slot, self._hit, self._ev = ctypes.c_int(), ctypes.c_int(), ctypes.c_int64()

    def __del__(self):
        try:
            if self.handle and _lib is not None:
                _lib.lora_slot_cache_destroy(ctypes.c_void_p(self.handle))
                self.handle = 0
        except Exception:
            pass

    def acquire(self, key: int, pin: bool = False):
        """-> (slot, hit, evicted_key or -1)."""
        _check("lora_slot_cache_acquire", _lib.lora_slot_cache_acquire(
            ctypes.c_void_p(self.handle), key, 1 if pin else 0, ctypes.byref(self._slot), ctypes.byref(self._hit),
            ctypes.byref(self._ev)))
        return self._slot.value, bool(self._hit.value), self._ev.value

    def unpin(self, slot: int) -> None:
        _check("lora_slot_cache_unpin", _lib.lora_slot_cache_unpin(ctypes.c_void_p(self.handle), slot))

    def invalidate(self, slot: int) -> None:
        _check("lora_slot_cache_invalidate", _lib.lora_slot_cache_invalidate(ctypes.c_void_p(self.handle), slot))

    def lookup(self, key: int) -> int:
        _check("lora_slot_cache_lookup", _lib.lora_slot_cache_lookup(ctypes.c_void_p(self.handle), key,
                                                                     ctypes.byref(self._slot)))
        return self._slot.value

    def stats(self):
        h, m, e = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check("lora_slot_cache_stats", _lib.lora_slot_cache_stats(ctypes.c_void_p(self.handle), ctypes.byref(h),
                                                                   ctypes.byref(m), ctypes.byref(e)))
        return h.value, m.value, e.value


def _refuse(name: str, why: str):
    raise LoraError(name, -1, why)


def _row_tensors(name: str, *tensors):
    """Check [T, heads, head_dim] tensors (None: absent): one device, rows whose
    elements are adjacent."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if t.dim() != 3 or not t.is_cuda or t.dtype not in DTYPES:
            _refuse(name, "row tensors are CUDA tensors [T, heads, head_dim] of bf16, fp16 or fp32")
        if t.stride(2) != 1 and t.shape[2] > 1:
            _refuse(name, "the elements of a row are adjacent")
        if dev is not None and t.device != dev:
            _refuse(name, "tensors on different devices")
        dev = t.device
    return dev


def _ints(name: str, dev, n, *tensors):
    """Check contiguous int32 tensors on `dev` with at least n elements (None: absent)."""
    for t in tensors:
        if t is None:
            continue
        if t.dtype != torch.int32 or t.device != dev or not t.is_contiguous() or t.numel() < n:
            _refuse(name, f"index arrays are contiguous int32 tensors on {dev} with at least {n} elements")


def _same(name: str, what: str, a, b):
    if a != b:
        _refuse(name, f"{what}: {tuple(a) if isinstance(a, torch.Size) else a} against {tuple(b) if isinstance(b, torch.Size) else b}")


def _r(t: Optional[torch.Tensor]):
    """lora_rows_t of a tensor (None: a null pointer)."""
    if t is None:
        return None
    n, s = t.shape, t.stride()   # the stride of a dimension of one element says nothing
    return ctypes.byref(LoraRows(t.data_ptr(), s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0))


def _kv(name: str, pages: torch.Tensor, kv_heads: int, head_dim: int, block_tokens: int):
    """lora_kv_cache_t over pages [num_pages, page bytes or values], rows contiguous."""
    if pages.dim() != 2 or not pages.is_cuda or not pages.is_contiguous():
        _refuse(name, "pages is a contiguous CUDA tensor [num_pages, page]")
    return ctypes.byref(LoraKvCache(pages.data_ptr(), pages.shape[1] * pages.element_size(), pages.shape[0], kv_heads,
                                    head_dim, block_tokens))


class _On:
    """Runs a call with the tensors' device current; stream None is that device's current stream."""

    def __init__(self, dev, stream):
        self.dev, self.stream = dev, stream

    def __enter__(self):
        self.back = torch.cuda.current_device()
        if self.dev.index != self.back:
            torch.cuda.set_device(self.dev)
        return _s(self.stream)

    def __exit__(self, *_):
        if self.dev.index != self.back:
            torch.cuda.set_device(self.back)


def lora_kv_block_bytes(kv_heads: int, head_dim: int, block_tokens: int) -> int:
    return int(load_library().lora_kv_block_bytes(kv_heads, head_dim, block_tokens))


def lora_kv_layout(past_len, new_len, req_ids, block_tokens: int, block_table, free_pages, free_head, cu_new, kv_len,
                   positions, slots, ids=None, free_head_out=None, err=None, stream=None) -> None:
    """past_len, new_len, req_ids [R], block_table [R, max_blocks]; cu_new [R + 1], kv_len [R], positions, slots, ids [T]
    out; free_pages None: block_table already names every block."""
    n = "lora_kv_layout"
    if block_table.dim() != 2 or positions.dim() != 1:
        _refuse(n, "block_table is [R, max_blocks], positions [T]")
    if not past_len.is_cuda:
        _refuse(n, "past_len is a CUDA tensor")
    R, T, dev = past_len.numel(), positions.numel(), past_len.device
    _ints(n, dev, R, past_len, new_len, req_ids, kv_len)
    _ints(n, dev, R + 1, cu_new)
    _ints(n, dev, R * block_table.shape[1], block_table)
    _ints(n, dev, T, positions, slots, ids)
    _ints(n, dev, 0, free_pages)
    _ints(n, dev, 1, err)
    _ints(n, dev, 1, free_head, free_head_out)
    with _On(dev, stream) as st:
        _check(n, load_library().lora_kv_layout(
            _p(past_len), _p(new_len), _p(req_ids), R, T, block_tokens, _p(block_table), block_table.shape[1],
            _p(free_pages), 0 if free_pages is None else free_pages.numel(), _p(free_head), _p(cu_new), _p(kv_len),
            _p(positions), _p(slots), _p(ids), _p(free_head_out), _p(err), st))


def _rope_args(name, q, k, v, positions, inv_freq, q_out, k_out, v_out, slots=None):
    dev = _row_tensors(name, q, k, v, q_out, k_out, v_out)
    first = k if q is None else q
    for x, y in ((q, q_out), (k, k_out), (v, v_out)):
        if x is not None and y is not None:
            _same(name, "input and output shapes", x.shape, y.shape)
        if x is not None:
            _same(name, "rows and head_dim", (x.shape[0], x.shape[2], x.dtype), (first.shape[0], first.shape[2], first.dtype))
    outs = [x.dtype for x in (q_out, k_out, v_out) if x is not None]
    if any(o != outs[0] for o in outs):
        _refuse(name, "outputs of different types")
    _ints(name, dev, first.shape[0], positions, slots)
    if inv_freq is not None and (inv_freq.dtype != torch.float32 or inv_freq.device != dev or not inv_freq.is_contiguous()):
        _refuse(name, f"inv_freq is a contiguous fp32 tensor on {dev}")
    return dev, first, DTYPES[outs[0] if outs else first.dtype]


def lora_rope(q, k, positions, inv_freq, q_out, k_out=None, interleaved: bool = False, mscale: float = 1.0,
              stream=None) -> None:
    """q [T, q_heads, head_dim] (k likewise, or None with k_out None); inv_freq [rot_dim / 2] fp32 on the device."""
    n = "lora_rope"
    dev, first, dst = _rope_args(n, q, k, None, positions, inv_freq, q_out, k_out, None)
    if (k is None) != (k_out is None):
        _refuse(n, "k and k_out come together")
    with _On(dev, stream) as st:
        _check(n, load_library().lora_rope(
            _r(q), q.shape[1], _r(k), 0 if k is None else k.shape[1], DTYPES[q.dtype], q.shape[0], q.shape[2],
            _p(positions), _p(inv_freq), 0 if inv_freq is None else 2 * inv_freq.numel(), int(interleaved), mscale,
            _r(q_out), _r(k_out), dst, st))


def lora_kv_append(q, k, v, positions, inv_freq, slots, pages, block_tokens: int, q_out, k_out=None, v_out=None,
                   interleaved: bool = False, mscale: float = 1.0, dtype=None, err=None, stream=None) -> None:
    """lora_rope on q and k, then k and v into the cache `pages` [num_pages, page].  dtype: the type that is cached and
    written, by default that of the outputs (of k when there is none)."""
    n = "lora_kv_append"
    dev, first, dst = _rope_args(n, q, k, v, positions, inv_freq, q_out, k_out, v_out, slots)
    _same(n, "k and v shapes", k.shape, v.shape)
    if (q is None) != (q_out is None):
        _refuse(n, "q and q_out come together")
    if dtype is not None:
        if any(x is not None and x.dtype != dtype for x in (q_out, k_out, v_out)):
            _refuse(n, "outputs of another type than dtype")
        dst = DTYPES[dtype]
    if pages.device != dev:
        _refuse(n, "pages on another device")
    _ints(n, dev, 1, err)
    kv = _kv(n, pages, k.shape[1], k.shape[2], block_tokens)
    with _On(dev, stream) as st:
        _check(n, load_library().lora_kv_append(
            _r(q), 0 if q is None else q.shape[1], _r(k), _r(v), DTYPES[k.dtype], k.shape[0], _p(positions), _p(inv_freq),
            0 if inv_freq is None else 2 * inv_freq.numel(), int(interleaved), mscale, _p(slots), kv, _r(q_out), _r(k_out),
            _r(v_out), dst, _p(err), st))


def lora_kv_gather(pages, block_tokens: int, slots, k_out, v_out=None, err=None, stream=None) -> None:
    """Rows slots[t] of the cache into k_out and v_out [T, kv_heads, head_dim] (either may be None)."""
    n = "lora_kv_gather"
    dev = _row_tensors(n, k_out, v_out)
    first = v_out if k_out is None else k_out
    if k_out is not None and v_out is not None:
        _same(n, "k_out and v_out", (k_out.shape, k_out.dtype), (v_out.shape, v_out.dtype))
    if pages.device != dev:
        _refuse(n, "pages on another device")
    _ints(n, dev, first.shape[0], slots)
    _ints(n, dev, 1, err)
    kv = _kv(n, pages, first.shape[1], first.shape[2], block_tokens)
    with _On(dev, stream) as st:
        _check(n, load_library().lora_kv_gather(kv, _p(slots), first.shape[0], _r(k_out), _r(v_out), DTYPES[first.dtype],
                                                _p(err), st))


def lora_kv_attend_workspace_size(q_heads: int, kv_heads: int, head_dim: int, max_q_len: int) -> int:
    return int(load_library().lora_kv_attend_workspace_size(q_heads, kv_heads, head_dim, max_q_len))


def _lse(name, lse, q):
    if lse is not None and (lse.dtype != torch.float32 or lse.device != q.device or not lse.is_contiguous() or
                            lse.shape != q.shape[:2]):
        _refuse(name, "lse is a contiguous fp32 tensor [T, q_heads] on the device of q")


def lora_kv_attend(q, pages, block_tokens: int, kv_heads: int, block_table, cu_q, kv_len, max_q_len: int, scale: float,
                   out, ws, lse=None, err=None, stream=None) -> None:
    """q, out [T, q_heads, head_dim]; block_table [R, max_blocks], cu_q [R + 1], kv_len [R]."""
    n = "lora_kv_attend"
    dev = _row_tensors(n, q, out)
    _same(n, "q and out", (q.shape, q.dtype), (out.shape, out.dtype))
    if pages.device != dev or ws.device != dev:
        _refuse(n, "pages or ws on another device")
    if block_table.dim() != 2:
        _refuse(n, "block_table is [R, max_blocks]")
    R, width = block_table.shape
    _ints(n, dev, R * width, block_table)
    _ints(n, dev, R, kv_len)
    _ints(n, dev, R + 1, cu_q)
    _ints(n, dev, 1, err)
    _lse(n, lse, q)
    kv = _kv(n, pages, kv_heads, q.shape[2], block_tokens)
    with _On(dev, stream) as st:
        _check(n, load_library().lora_kv_attend(
            _r(q), q.shape[0], q.shape[1], DTYPES[q.dtype], kv, _p(block_table), width, _p(cu_q), _p(kv_len), R, max_q_len,
            scale, _r(out), _p(lse), _p(ws), ws.numel() * ws.element_size(), _p(err), st))


def lora_prompt_attend(q, k, v, cu_q, cu_k, scale: float, out, lse=None, err=None, stream=None) -> None:
    """q, out [Tq, q_heads, head_dim], k, v [Tk, kv_heads, head_dim]; cu_q, cu_k [R + 1]."""
    n = "lora_prompt_attend"
    dev = _row_tensors(n, q, k, v, out)
    _same(n, "q and out", (q.shape, q.dtype), (out.shape, out.dtype))
    _same(n, "k and v", (k.shape, k.dtype), (v.shape, v.dtype))
    _same(n, "q and k", (q.shape[2], q.dtype), (k.shape[2], k.dtype))
    _ints(n, dev, 2, cu_q, cu_k)
    _same(n, "cu_q and cu_k", cu_q.numel(), cu_k.numel())
    _ints(n, dev, 1, err)
    _lse(n, lse, q)
    with _On(dev, stream) as st:
        _check(n, load_library().lora_prompt_attend(
            _r(q), _r(k), _r(v), q.shape[0], k.shape[0], q.shape[1], k.shape[1], q.shape[2], DTYPES[q.dtype], _p(cu_q),
            _p(cu_k), cu_q.numel() - 1, scale, _r(out), _p(lse), _p(err), st))


def lora_set_option(key: int, value: int) -> None:
    _check("lora_set_option", load_library().lora_set_option(key, value))


def lora_get_option(key: int) -> int:
    return int(load_library().lora_get_option(key))


def lora_last_cuda_error() -> str:
    return load_library().lora_last_cuda_error().decode()


def lora_last_launch_count() -> int:
    return int(load_library().lora_last_launch_count())
