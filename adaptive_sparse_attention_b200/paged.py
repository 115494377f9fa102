"""Torch-facing binding of the paged key-value cache: page tables, cache append, and alpha-entmax
attention of one new token per request.  Argument marshalling only, as in api.py.

A cache is two tensors k_cache, v_cache [num_pages, Hkv, page_size, d] of one dtype (float32 or
bfloat16), shape and strides with a unit-stride last dimension; a cache stored with tokens before
heads is passed as its transposed view.  A server's step:

    slots, lens, cu_new, free_start = page_tables(lens, new_lens, free_pages, free_start,
                                                  block_tables, page_size, n_new)
    paged_append(k, v, k_cache, v_cache, slots)
    out, tau = entmax_attn_decode(q, k_cache, v_cache, block_tables, lens, alpha)

The calls run on the device of their tensors, on `stream` (default: that device's current stream);
outputs and scratch memory that they allocate belong to that stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import _native as N
from .api import _DT


def _require(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _int32(t, name: str, dim: int, dev) -> None:
    if not (t.dtype is torch.int32 and t.dim() == dim and t.is_cuda and
            (t.numel() == 0 or t.stride(-1) == 1 or t.shape[-1] == 1)):
        raise ValueError(f"{name} must be a {dim}-D int32 CUDA tensor with a unit-stride last "
                         "dimension")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")


@contextlib.contextmanager
def _elsewhere(dev, stream):
    """Makes `dev` and `stream` current."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(
                    stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream), dev)
            with torch.cuda.stream(stream):
                yield


def _call(fn, dev, stream):
    """fn(raw stream) with the device and stream current, so that it allocates for them too."""
    if stream is None and torch.cuda.current_device() == dev.index:
        return fn(torch.cuda.current_stream(dev).cuda_stream)
    with _elsewhere(dev, stream):
        return fn(torch.cuda.current_stream(dev).cuda_stream)


def _cache_dims(k_cache, v_cache):
    """(num_pages, Hkv, page_size, d) and the strides of a checked cache."""
    if not (k_cache.dim() == 4 and k_cache.is_cuda and k_cache.dtype in _DT and
            k_cache.stride(3) == 1):
        raise ValueError("k_cache must be a float32 or bfloat16 CUDA tensor [num_pages, Hkv, "
                         "page_size, d] with a unit-stride last dimension")
    shape, strides = k_cache.shape, k_cache.stride()
    if v_cache.shape != shape or v_cache.stride() != strides or \
            v_cache.dtype != k_cache.dtype or v_cache.device != k_cache.device:
        raise ValueError("v_cache must have the shape, strides, dtype and device of k_cache")
    if 0 in shape:
        raise ValueError("the cache is empty")
    # a dimension of one element may carry any stride: give the library one that it accepts
    d = shape[3]
    return shape, [s if n > 1 else max(s // 8 * 8, d) for n, s in zip(shape[:3], strides)]


def page_tables(lens, new_lens, free_pages, free_start, block_tables, page_size: int, n_new: int,
                padded: bool = False, slots=None, lens_out=None, cu_new=None, free_next=None,
                stream=None):
    """Grows the block tables for new_lens[b] new tokens of request b, which holds lens[b], from
    the free list, and maps every new token to its slot (page * page_size + position in the page).

    lens, new_lens int32 [B]; free_pages int32 [n_free], of which the first free_start (int32 [1])
    are taken; block_tables int32 [B, W], new entries written in place.  Returns (slots, lens_out,
    cu_new, free_next): slots int64 [n_new], the new tokens packed in request order and -1 behind
    the last, or with padded=True [B, n_new], -1 for t >= new_lens[b]; lens_out int32 [B]; cu_new
    int32 [B + 1], the prefix sums of new_lens (the cu_seqlens of the packed forward pass); free_next
    int32 [1].  A request that does not fit keeps its length and gets slots of -1 (see
    include/entmax_attn.h).  The outputs may be given; lens_out and free_next may not be the
    inputs themselves."""
    dev = lens.device
    _int32(lens, "lens", 1, dev)
    _int32(new_lens, "new_lens", 1, dev)
    _int32(free_pages, "free_pages", 1, dev)
    _int32(free_start, "free_start", 1, dev)
    _int32(block_tables, "block_tables", 2, dev)
    B, W = block_tables.shape
    _require(lens.shape[0] == B and new_lens.shape[0] == B and free_start.shape[0] == 1,
             "lens and new_lens must be [B], free_start [1], block_tables [B, W]")

    def go(raw):
        shape = (B, n_new) if padded else (n_new,)
        s = torch.empty(shape, dtype=torch.int64, device=dev) if slots is None else slots
        lo = torch.empty_like(lens) if lens_out is None else lens_out
        cu = torch.empty(B + 1, dtype=torch.int32, device=dev) if cu_new is None else cu_new
        nx = torch.empty_like(free_start) if free_next is None else free_next
        if slots is not None:
            _require(s.shape == shape and s.dtype == torch.int64 and s.is_contiguous() and
                     s.device == dev, "slots must be contiguous int64 [n_new], padded: [B, n_new]")
        for t, n, name in ((lo, B, "lens_out"), (cu, B + 1, "cu_new"), (nx, 1, "free_next")):
            _int32(t, name, 1, dev)
            _require(t.shape[0] == n, f"{name} must have {n} elements")
        rc = N.lib().entmax_attn_page_tables(
            lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), free_pages.shape[0],
            free_start.data_ptr(), block_tables.data_ptr(), block_tables.stride(0) if B > 1 else W, W, B,
            page_size, s.data_ptr(), n_new, 1 if padded else 0, lo.data_ptr(), cu.data_ptr(),
            nx.data_ptr(), raw)
        N.check(rc, "entmax_attn_page_tables")
        return s, lo, cu, nx

    return _call(go, dev, stream)


def paged_append(k, v, k_cache, v_cache, slots, stream=None) -> None:
    """Stores new tokens' keys and values in the slots given by page_tables.  k, v [B, Hkv, T, d]
    or packed [Hkv, N, d], one dtype with the cache, any strides in multiples of 16 bytes with a
    unit-stride last dimension; slots int64 [B, T] or [B * T] (packed: [N]), negative ones are
    skipped.  The slots must differ from one another."""
    (pages, Hkv, P, d), (ps, hs, ss) = _cache_dims(k_cache, v_cache)
    dev = k_cache.device
    if k.dim() == 4:
        B, H, T, dk = k.shape
        sb, sh, st, se = k.stride()
    elif k.dim() == 3:
        (H, T, dk), (sh, st, se) = k.shape, k.stride()
        B, sb = 1, 0
    else:
        raise ValueError("k must be [B, Hkv, T, d] or packed [Hkv, N, d]")
    _require(H == Hkv and dk == d and k.dtype == k_cache.dtype and k.device == dev and se == 1,
             "k must have the cache's heads, head size, dtype and device, and unit-stride rows")
    _require(v.shape == k.shape and v.stride() == k.stride() and v.dtype == k.dtype and
             v.device == dev, "v must have the shape, strides, dtype and device of k")
    _require(slots.dtype is torch.int64 and slots.device == dev and slots.is_contiguous() and
             slots.numel() == B * T, "slots must be a contiguous int64 tensor, one per new token")
    if B * T == 0:
        return

    def go(raw):
        rc = N.lib().entmax_attn_paged_append(
            k.data_ptr(), v.data_ptr(), sb if B > 1 else 0, sh if H > 1 else 0, st if T > 1 else 0,
            k_cache.data_ptr(), v_cache.data_ptr(), ps, hs, ss, pages, P, slots.data_ptr(), B, H,
            T, d, _DT[k.dtype], raw)
        N.check(rc, "entmax_attn_paged_append")

    _call(go, dev, stream)


def decode_workspace_bytes(B: int, Hq: int, Hkv: int, max_len: int) -> int:
    return int(N.lib().entmax_attn_decode_workspace_bytes(B, Hq, Hkv, max_len))


def alloc_decode_workspace(q, k_cache, max_len: int):
    """Workspace of entmax_attn_decode for q's batch and requests of up to max_len tokens."""
    n = decode_workspace_bytes(q.shape[0], q.shape[1], k_cache.shape[1], max_len)
    _require(n > 0, "bad sizes for a decode workspace")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def entmax_attn_decode(q, k_cache, v_cache, block_tables, seq_lens, alpha: float = 1.5,
                       n_iter: int = 10, max_len: int | None = None, out=None, tau=None,
                       workspace=None, stream=None):
    """alpha-entmax attention of one new token per request over its seq_lens[b] cached keys.

    q [B, Hq, d] or [B, Hq, 1, d] in the cache's dtype, unit-stride rows, batch and head strides in
    multiples of 16 bytes; block_tables int32 [B, W]; seq_lens int32 [B], at most max_len (default:
    W * page_size; a smaller bound needs less workspace).  Returns (out, tau): out like q, tau fp32
    with q's leading shape.  A request of length 0 gets out = 0 and tau = +inf.  workspace: a uint8
    buffer of decode_workspace_bytes(B, Hq, Hkv, max_len), allocated here unless given; calls that
    overlap on the device need one each."""
    (pages, Hkv, P, d), (ps, hs, ss) = _cache_dims(k_cache, v_cache)
    dev = k_cache.device
    _require((q.dim() == 3 or (q.dim() == 4 and q.shape[2] == 1)) and q.shape[-1] == d and
             q.dtype == k_cache.dtype and q.device == dev and q.stride(-1) == 1,
             "q must be [B, Hq, d] or [B, Hq, 1, d] with the cache's head size, dtype and device, "
             "and unit-stride rows")
    B, Hq = q.shape[:2]
    _int32(block_tables, "block_tables", 2, dev)
    _int32(seq_lens, "seq_lens", 1, dev)
    W = block_tables.shape[1]
    _require(block_tables.shape[0] == B and seq_lens.shape[0] == B and W > 0,
             "block_tables must be [B, W] and seq_lens [B]")
    if max_len is None:
        max_len = W * P

    def go(raw):
        o = torch.empty(q.shape, dtype=q.dtype, device=dev) if out is None else out
        t = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev) if tau is None else tau
        ws = alloc_decode_workspace(q, k_cache, max_len) if workspace is None else workspace
        if out is not None:
            _require(o.shape == q.shape and o.dtype == q.dtype and o.is_contiguous() and
                     o.device == dev, "out must be contiguous, with q's shape, dtype and device")
        if tau is not None:
            _require(t.shape == q.shape[:-1] and t.dtype == torch.float32 and
                     t.is_contiguous() and t.device == dev,
                     "tau must be contiguous float32 with q's leading shape")
        if workspace is not None:
            _require(ws.device == dev and ws.is_contiguous(),
                     "workspace must be a contiguous buffer on the cache's device")
        rc = N.lib().entmax_attn_decode(
            q.data_ptr(), q.stride(0) if B > 1 else 0, q.stride(1) if Hq > 1 else 0,
            k_cache.data_ptr(), v_cache.data_ptr(), ps, hs, ss, pages, P, block_tables.data_ptr(),
            block_tables.stride(0) if B > 1 else W, W, seq_lens.data_ptr(), o.data_ptr(), t.data_ptr(),
            ws.data_ptr(), ws.numel() * ws.element_size(), B, Hq, Hkv, max_len, d, float(alpha),
            int(n_iter), _DT[q.dtype], raw)
        N.check(rc, "entmax_attn_decode")
        return o, t

    return _call(go, dev, stream)
