"""The paged key/value cache: serving counterpart of the jagged forward.

* ``paged_cache(n_pages, page_size, H, D, format=..., device=...)``: page
  buffers for keys and values, in bf16 or MXFP8 (E4M3 codes, one E8M0 exponent
  per 32 neighbouring values of a row); ``PagedCache(k, v, k_scales, v_scales)``
  wraps buffers that exist already.
* ``cache_append(cache, k, v, page_table, start, off=..., rope=...)``: writes
  new jagged rows, quantising and rotating them on the way.
* ``cache_read(cache, page_table, off, start=..., total=...)``: cached rows as
  jagged bf16 K and V, for ``forward`` / ``attention``.
* ``decode(q, cache, page_table, kv_lens, q_off=..., ...)``: attention of one
  or a few new query rows per sequence over the cache, with ``forward``'s
  activations and masks; query heads may share key/value heads.
* ``page_pool(n_pages, page_size)``: the cache's free pages, in device memory;
  ``page_assign(pool, page_table, start, off=...)`` gives sequences the pages
  that new rows need (before ``cache_append``) and returns the rows' slots,
  ``page_release(pool, page_table, lens, keep=...)`` takes pages back, both without
  a host round trip.

Row ``pos`` of sequence b lies in page ``page_table[b, pos // page_size]``.
Every tensor lies on the cache's device; calls run on that device's current
stream and allocate only their outputs and scratch (from PyTorch's allocator, so
calls on several streams, and captured graphs, do not share any). Rows that a call
leaves as they were (padding behind the last sequence, skipped sequences) hold
anything in outputs that the call itself allocates. Device-side errors (a bad
page, a length past the table) are read with ``device_status``.
"""
from __future__ import annotations

import ctypes

import torch

from . import SOFTMAX, _act, _mask, _width
from . import _binding as B

_FORMATS = {"bf16": B.CACHE_BF16, "mxfp8": B.CACHE_MXFP8}

# One 256-byte status word per device, kept for the life of the process
# (captured graphs hold its address).
_status_blocks: dict = {}


def status_block(index: int) -> torch.Tensor:
    t = _status_blocks.get(index)
    if t is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the first paged-cache or row-operator call on a device cannot be captured into a graph; "
                               "make one call before the capture")
        t = torch.zeros(256, dtype=torch.uint8, device=torch.device("cuda", index))
        torch.cuda.current_stream(index).synchronize()
        t = _status_blocks.setdefault(index, t)
    return t


def status_address(index: int) -> int:
    return status_block(index).data_ptr()


class PagedCache:
    """Page buffers k, v [n_pages, H, page_size, D] (bf16, or uint8 E4M3 codes with uint8 E8M0 exponents k_scales,
    v_scales [n_pages, H, page_size, D/32]); the layout is jattn_cache_t's. Holds the tensors it is given."""

    __slots__ = ("_k", "_v", "_k_scales", "_v_scales", "_c", "_ref", "_device", "_index", "_page", "_H", "_D")

    def __init__(self, k, v, k_scales=None, v_scales=None):
        mx = k_scales is not None
        if k.dim() != 4 or k.shape != v.shape or not k.is_cuda or v.device != k.device:
            raise ValueError("k and v must be CUDA tensors [n_pages, H, page_size, D] of one shape and device")
        want = torch.uint8 if mx else torch.bfloat16
        if k.dtype != want or v.dtype != want or (v_scales is not None) != mx:
            raise ValueError("k and v must both be bf16 without scales, or uint8 codes with k_scales and v_scales")
        n, H, page, D = k.shape
        if D not in (64, 128) or page < 8 or page > 4096 or page & (page - 1):
            raise ValueError("D must be 64 or 128 and page_size a power of two from 8 to 4096")
        for t in (k_scales, v_scales) if mx else ():
            if t.dtype != torch.uint8 or tuple(t.shape) != (n, H, page, D // 32) or t.device != k.device:
                raise ValueError("scales must be uint8 [n_pages, H, page_size, D/32] on the cache's device")
        if not all(t.is_contiguous() for t in (k, v, k_scales, v_scales) if t is not None):
            raise ValueError("cache buffers must be contiguous")
        if k.requires_grad or v.requires_grad:
            raise ValueError("cache buffers take no gradient: pass detached tensors")
        self._k, self._v, self._k_scales, self._v_scales = k, v, k_scales, v_scales
        self._c = B.cache(n, page, H, D, B.CACHE_MXFP8 if mx else B.CACHE_BF16, k, v, k_scales, v_scales)
        self._ref = ctypes.byref(self._c)
        self._device, self._index, self._page, self._H, self._D = k.device, k.device.index, page, H, D

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scales = property(lambda self: self._k_scales)
    v_scales = property(lambda self: self._v_scales)
    n_pages = property(lambda self: self._c.n_pages)
    page_size = property(lambda self: self._page)
    H = property(lambda self: self._H)
    D = property(lambda self: self._D)
    format = property(lambda self: "mxfp8" if self._c.format == B.CACHE_MXFP8 else "bf16")
    device = property(lambda self: self._device)


def paged_cache(n_pages, page_size, H, D, format="bf16", device="cuda") -> PagedCache:
    """A new cache of ``n_pages`` zeroed pages of ``page_size`` rows (a power of two, 8 to 4096)."""
    if format not in _FORMATS:
        raise ValueError(f"format must be one of {sorted(_FORMATS)}")
    mx = format == "mxfp8"
    shape = (n_pages, H, page_size, D)
    k, v = (torch.zeros(shape, dtype=torch.uint8 if mx else torch.bfloat16, device=device) for _ in range(2))
    if not mx:
        return PagedCache(k, v)
    ks, vs = (torch.zeros((*shape[:3], D // 32), dtype=torch.uint8, device=device) for _ in range(2))
    return PagedCache(k, v, ks, vs)


class PagePool:
    """Free pages of a cache with pages of ``page_size`` rows: free_pages int32 [n_pages], of which the first count[0] (int64
    [1]) are a stack of free pages, the next one to be taken last. Holds the tensors it is given. Calls on one pool follow
    each other (one stream, or events between streams), as those on a cache do."""

    __slots__ = ("_free", "_count", "_page")

    def __init__(self, free_pages, count, page_size):
        if free_pages.dtype is not torch.int32 or free_pages.dim() != 1 or not free_pages.is_cuda \
                or free_pages.numel() == 0 or not free_pages.is_contiguous():
            raise ValueError("free_pages must be a contiguous CUDA int32 tensor [n_pages]")
        if count.dtype is not torch.int64 or count.shape != (1,) or count.device != free_pages.device:
            raise ValueError("count must be an int64 tensor [1] on the device of free_pages")
        if page_size < 1 or page_size > 4096 or page_size & (page_size - 1):
            raise ValueError("page_size must be a power of two from 1 to 4096")
        self._free, self._count, self._page = free_pages, count, int(page_size)

    free_pages = property(lambda self: self._free)
    count = property(lambda self: self._count)
    n_pages = property(lambda self: self._free.numel())
    page_size = property(lambda self: self._page)
    device = property(lambda self: self._free.device)


def page_pool(n_pages, page_size, device="cuda") -> PagePool:
    """A pool whose ``n_pages`` pages are all free; page 0 is taken first."""
    free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)
    return PagePool(free, torch.full((1,), n_pages, dtype=torch.int64, device=device), page_size)


def _check_rows(cache, x, name):
    if x.dtype is not torch.bfloat16 or x.dim() != 3 or x.device != cache._device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 tensor [total, H, D] on the cache's device")


def _check_no_grad(*outputs):
    for x in outputs:
        if x is not None and x.requires_grad and torch.is_grad_enabled():
            raise ValueError("outputs are written without a gradient: pass tensors that need none")


def _check_index(cache, t, n, name):
    if t.dtype is not torch.int64 or t.shape != (n,) or t.device != cache._device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int64 tensor [{n}] on the cache's device")


def _check_table(cache, t):
    if t.dtype is not torch.int32 or t.dim() != 2 or t.device != cache._device or not t.is_contiguous() \
            or t.numel() == 0:
        raise ValueError("page_table must be a contiguous int32 tensor [B, max_pages] on the cache's device")


def _check_rope(cache, rope):
    cos, sin = rope
    for t in rope:
        if t.dtype is not torch.float32 or t.dim() != 2 or t.shape[1] != cache._D // 2 or t.shape != cos.shape \
                or t.device != cache._device or not t.is_contiguous():
            raise ValueError("rope tables must be two contiguous fp32 tensors [rows, D/2] on the cache's device")
    return cos, sin


def _launch(cache, fn, *args):
    """fn(*args, workspace, its bytes, stream) with the cache's device current."""
    index = cache._index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _launch(cache, fn, *args)
    fn(*args, status_block(index).data_ptr(), 256, torch._C._cuda_getCurrentRawStream(index))


def cache_append(cache, k, v, page_table, start, off=None, rope=None):
    """Write rows k, v [total, H, D] bf16 into the cache: row i of sequence b
    at position start[b] + i (start int64 [B], the length cached before; negative
    skips the sequence). ``off`` int64 [B+1] are the rows' prefix sums (None: one
    row per sequence); rows behind off[B] are skipped. With ``rope`` = (cos, sin)
    tables keys are rotated at their own positions before they are stored. No
    gradient. See jattn_cache_append."""
    _check_table(cache, page_table)
    nb = page_table.shape[0]
    _check_rows(cache, k, "k")
    _check_rows(cache, v, "v")
    if (k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
        raise ValueError("cache_append has no backward pass: call it under torch.no_grad() or on detached rows")
    total = k.shape[0]
    if k.shape != v.shape or k.shape != (total, cache._H, cache._D):
        raise ValueError("k and v must be [total, H, D] with the cache's H and D")
    _check_index(cache, start, nb, "start")
    if off is not None:
        _check_index(cache, off, nb + 1, "off")
    elif total != nb:
        raise ValueError("without off there must be one row per sequence")
    cos, sin = _check_rope(cache, rope) if rope is not None else (None, None)
    _launch(cache, B.cache_append, cache._ref, nb, total, off, start, page_table, k, v, cos, sin)


def cache_read(cache, page_table, off, start=None, total=None, k=None, v=None):
    """Cached rows as jagged bf16 tensors (k, v) [total, H, D]: row i of
    sequence b (off int64 [B+1]) is position start[b] + i (start int64 [B], None: 0;
    negative leaves the sequence's rows as they were). ``total`` defaults to
    off[-1] (a host read) or to the rows of the given outputs. See jattn_cache_read."""
    _check_table(cache, page_table)
    nb = page_table.shape[0]
    _check_index(cache, off, nb + 1, "off")
    if start is not None:
        _check_index(cache, start, nb, "start")
    for x, name in ((k, "k"), (v, "v")):
        if x is not None:
            _check_rows(cache, x, name)
            total = x.shape[0] if total is None else total
            if x.shape != (total, cache._H, cache._D):
                raise ValueError(f"{name} must be [total, H, D] with the cache's H and D")
    _check_no_grad(k, v)
    total = int(off[-1].item()) if total is None else int(total)
    k = k if k is not None else torch.empty((total, cache._H, cache._D), dtype=torch.bfloat16, device=cache._device)
    v = v if v is not None else torch.empty_like(k)
    _launch(cache, B.cache_read, cache._ref, nb, total, off, start, page_table, k, v)
    return k, v


def decode(q, cache, page_table, kv_lens, q_off=None, act="softmax", causal=False, window=0, scale=None,
           norm_by_lkv=False, block=0, max_kv=None, out=None, lse=None):
    """Attention of new query rows q [total_q, Hq, D] bf16 over the cache.
    Returns (O [total_q, Hq, D] bf16, LSE [total_q, Hq] fp32 or None).

    kv_lens int64 [B]: cached rows of each sequence, the new ones included;
    q_off int64 [B+1]: the query rows' prefix sums (None: one row each), the last
    row of a sequence standing at its last cached position. Hq is a multiple of
    the cache's H. Activations, masks and scale as in ``forward``. ``max_kv``
    bounds kv_lens (default: the table's rows). Rows behind q_off[B] are left as
    they were in ``out`` / ``lse``. Weights meet the values as two bf16 parts, or on an
    MXFP8 cache as one fp16 number. No gradient. See jattn_decode."""
    _check_table(cache, page_table)
    nb, max_pages = page_table.shape
    _check_rows(cache, q, "q")
    if q.requires_grad and torch.is_grad_enabled():
        raise ValueError("decode has no backward pass: call it under torch.no_grad() or on a detached q")
    total_q, Hq, D = q.shape
    if D != cache._D or Hq == 0 or Hq % cache._H:
        raise ValueError("q must have the cache's D and a multiple of its heads")
    _check_index(cache, kv_lens, nb, "kv_lens")
    if q_off is not None:
        _check_index(cache, q_off, nb + 1, "q_off")
    elif total_q != nb:
        raise ValueError("without q_off there must be one query row per sequence")
    rows = max_pages * cache._page
    if max_kv is not None and not 0 <= max_kv <= rows:
        raise ValueError("max_kv must lie between 0 and the rows of the page table")
    a, mask = _act(act), _mask(causal, window, block)
    p = ctypes.byref(B.params(nb, total_q, rows if max_kv is None else max_kv, Hq, D, a, mask, _width(window, block),
                              scale, norm_by_lkv))
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    else:
        _check_rows(cache, out, "out")
    if a != SOFTMAX:
        lse = None
    elif lse is None:
        lse = torch.empty((total_q, Hq), dtype=torch.float32, device=cache._device)
    elif lse.dtype != torch.float32 or lse.shape != (total_q, Hq) or lse.device != q.device \
            or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [total_q, Hq] on the cache's device")
    _check_no_grad(out, lse)
    n = B.decode_scratch_size(p, cache._ref)
    scratch = torch.empty(n, dtype=torch.uint8, device=cache._device)
    _launch(cache, B.decode, p, cache._ref, q_off, kv_lens, page_table, q, out, lse, scratch.data_ptr(), n)
    return out, lse


def page_assign(pool, page_table, start, off=None, total=None, slots=True):
    """Give every sequence the pages that its new rows need: rows start[b] .. start[b] + n - 1 (start int64 [B], the rows
    before, whose pages page_table holds already; negative skips the sequence), n from the prefix sums ``off`` int64 [B+1] (None:
    one row each). Page numbers are written into page_table int32 [B, max_pages] where they are missing. Returns the new
    rows' slots int64 [total], page * page_size + place in the page (-1 for rows without one and rows behind off[B]);
    ``slots`` may be a tensor to write them to, or False for none: the cache's own calls find rows by page_table, slots are for
    a program's own kernels and buffers [n_pages * page_size, ...], and a large call is faster without. ``total`` defaults to off[-1] (a host read) or the rows
    of ``slots``. Where the pool has too few pages none is assigned (``device_status``). See jattn_page_assign."""
    if off is not None and total is None and not isinstance(slots, torch.Tensor):
        total = int(off[-1].item())
    return (B._host or B.host()).page_assign(pool._free, pool._count, pool._page, page_table, start, off,
                                             -1 if total is None else total, slots)


def page_release(pool, page_table, lens, keep=None):
    """Take back the pages of rows keep[b] .. lens[b] - 1 (int64 [B]; keep None: all rows, negative: the sequence is left as it
    is) that hold none of the rows kept; their entries in page_table become -1. The next page_assign takes them first, the first sequence's first
    page before all others. See jattn_page_release."""
    (B._host or B.host()).page_release(pool._free, pool._count, pool._page, page_table, lens, keep)
