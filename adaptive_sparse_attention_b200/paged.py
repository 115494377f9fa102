"""Paged key-value cache on torch tensors: page tables, cache append, and alpha-entmax attention of
one new token per request.  Checks, output allocation and the library call are in the compiled
binding (csrc/paged_binding.cpp, built to _paged.so); there is no fallback.

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

import torch

from . import _native as N

_binding = None


def _load():
    """The binding (loaded once, after the library it is linked to)."""
    global _binding
    if _binding is None:
        N.lib()
        try:
            from . import _paged
        except ImportError as e:
            raise N.NativeLibraryError(
                "the paged-cache binding is missing; build it with "
                f"`python -m adaptive_sparse_attention_b200.build` ({e})") from e
        _binding = _paged
    return _binding


def _on(stream, dev):
    """A context that makes `stream` (a torch stream or a raw handle) of `dev` current."""
    if isinstance(stream, torch.cuda.Stream) and stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {dev}")
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        # torch takes an external handle of 0 for none given and makes a new stream
        stream = torch.cuda.ExternalStream(raw, dev) if raw else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


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
    int32 [1].  B is at least 1; n_new may be 0.  A request that does not fit keeps its length and
    gets slots of -1 (see include/entmax_attn.h).  The outputs may be given; lens_out and free_next
    may not be the inputs themselves.  Where none of lens_out, cu_new and free_next is, they share
    one storage."""
    if stream is not None:
        with _on(stream, lens.device):
            return page_tables(lens, new_lens, free_pages, free_start, block_tables, page_size,
                               n_new, padded, slots, lens_out, cu_new, free_next)
    r = (_binding or _load()).page_tables(lens, new_lens, free_pages, free_start, block_tables,
                                          page_size, n_new, padded, slots, lens_out, cu_new,
                                          free_next)
    if type(r) is int:
        N.check(r, "entmax_attn_page_tables")
    return r


def paged_append(k, v, k_cache, v_cache, slots, stream=None) -> None:
    """Stores new tokens' keys and values in the slots given by page_tables.  k, v [B, Hkv, T, d]
    or packed [Hkv, N, d], one dtype with the cache, any strides in multiples of 16 bytes with a
    unit-stride last dimension; slots int64 [B, T] or [B * T] (packed: [N]), negative ones are
    skipped.  The slots must differ from one another."""
    if stream is not None:
        with _on(stream, k_cache.device):
            return paged_append(k, v, k_cache, v_cache, slots)
    r = (_binding or _load()).paged_append(k, v, k_cache, v_cache, slots)
    if r is not None:
        N.check(r, "entmax_attn_paged_append")


def decode_workspace_bytes(B: int, Hq: int, Hkv: int, max_len: int) -> int:
    return int(N.lib().entmax_attn_decode_workspace_bytes(B, Hq, Hkv, max_len))


def alloc_decode_workspace(q, k_cache, max_len: int):
    """Workspace of entmax_attn_decode for q's batch and requests of up to max_len tokens."""
    n = decode_workspace_bytes(q.shape[0], q.shape[1], k_cache.shape[1], max_len)
    if n == 0 and q.shape[0] != 0 and max_len != 0:  # without requests or keys none is needed
        raise ValueError("bad sizes for a decode workspace")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def entmax_attn_decode(q, k_cache, v_cache, block_tables, seq_lens, alpha: float = 1.5,
                       n_iter: int = 10, max_len: int | None = None, out=None, tau=None,
                       workspace=None, stream=None):
    """alpha-entmax attention of one new token per request over its seq_lens[b] cached keys.

    q [B, Hq, d] or [B, Hq, 1, d] in the cache's dtype, unit-stride rows, batch and head strides in
    multiples of 16 bytes; block_tables int32 [B, W]; seq_lens int32 [B], at most max_len (default:
    W * page_size; a smaller bound needs less workspace; 0 where all rows are unused).  n_iter is
    checked but has no effect (the forward pass's parameter): tau is searched until it has settled.
    Returns (out, tau): out like q, tau fp32 with q's leading shape.  A request of length 0 gets
    out = 0 and tau = +inf.  workspace: a buffer of decode_workspace_bytes(B, Hq, Hkv, max_len),
    allocated here unless given; calls that overlap on the device need one each."""
    if stream is not None:
        with _on(stream, k_cache.device):
            return entmax_attn_decode(q, k_cache, v_cache, block_tables, seq_lens, alpha, n_iter,
                                      max_len, out, tau, workspace)
    r = (_binding or _load()).decode(q, k_cache, v_cache, block_tables, seq_lens, alpha, n_iter,
                                     max_len, out, tau, workspace)
    if type(r) is int:
        N.check(r, "entmax_attn_decode")
    return r
