"""The paged-cache operators at the edges of what they accept: steps without tokens, keys or
requests."""
import random

import numpy as np
import pytest
import torch

import adaptive_sparse_attention_b200 as ea
from adaptive_sparse_attention_b200 import _native
from oracle import paged

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def check_tables(lens, new, free, start, tables, page, n_new, padded, **kw):
    want = paged.page_tables(lens, new, free, start, tables.cpu().numpy(), page, n_new, padded)
    got = ea.page_tables(i32(lens), i32(new), i32(free), i32([start]), tables, page, n_new, padded,
                         **kw)
    for name, a, b in zip(("tables", "slots", "lens", "cu", "next"), want, (tables,) + got):
        assert tuple(b.shape) in (np.shape(a), (1,)), name
        assert np.array_equal(a, b.cpu().numpy().reshape(np.shape(a))), name
    return got


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("B", [1, 5, 1000])
def test_tables_of_a_step_without_tokens(B, padded):
    """n_new = 0: lengths, offsets and the start are passed on; a request with new tokens all the
    same does not fit."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 40, size=B)
    tables = i32(rng.integers(0, 99, size=(B, 4)))
    before = tables.clone()
    for new in (np.zeros(B, dtype=int), (rng.random(B) < 0.5).astype(int)):
        check_tables(lens, new, [4, 5, 6], 1, tables, 16, 0, padded)
        check_tables(lens, new, [4, 5, 6], 1, tables, 16, 0, padded,
                     slots=torch.empty((B, 0) if padded else 0, dtype=torch.int64, device="cuda"))
    assert torch.equal(tables, before)


def unused_batch(B, Hq, Hkv, d, dtype, W=3):
    q = torch.randn(B, Hq, d).to(DT[dtype]).cuda()
    kc, vc = (torch.randn(4, Hkv, 16, d).to(DT[dtype]).cuda() for _ in range(2))
    return q, kc, vc, i32(np.full((B, W), -1)), i32([0] * B)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hq,Hkv,d", [(1, 1, 1, 64), (3, 40, 2, 128), (700, 8, 8, 64)])
@pytest.mark.parametrize("given", [False, True])
def test_decode_of_a_batch_of_unused_rows(dtype, B, Hq, Hkv, d, given):
    """max_len = max(seq_lens) = 0, with a workspace or without."""
    q, kc, vc, tables, lens = unused_batch(B, Hq, Hkv, d, dtype)
    ws = ea.alloc_decode_workspace(q, kc, 0) if given else None
    out, tau = ea.entmax_attn_decode(q, kc, vc, tables, lens, 1.5, max_len=0, workspace=ws)
    assert out.shape == q.shape and (out == 0).all()
    assert torch.isposinf(tau).all()
    assert ea.status() == 0


def test_decode_reports_a_length_above_a_bound_of_zero():
    q, kc, vc, tables, lens = unused_batch(4, 2, 1, 64, "bf16")
    tables[2, 0] = 1
    lens[2] = 1
    lens[3] = -1
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    out, tau = ea.entmax_attn_decode(q, kc, vc, tables, lens, 1.5, max_len=0, workspace=ws)
    assert ea.status() == _native.ERANGE and ea.status() == 0
    assert torch.isnan(out[2:]).all() and torch.isnan(tau[2:]).all()
    assert (out[:2] == 0).all() and torch.isposinf(tau[:2]).all()


def test_decode_of_no_requests():
    q, kc, vc, tables, lens = unused_batch(0, 4, 2, 64, "bf16")
    for x in (q, q.unsqueeze(2)):
        out, tau = ea.entmax_attn_decode(x, kc, vc, tables, lens, 1.5,
                                         workspace=ea.alloc_decode_workspace(x, kc, 48))
        assert out.shape == x.shape and tau.shape == x.shape[:-1] and tau.dtype == torch.float32
    with pytest.raises(ValueError):
        ea.entmax_attn_decode(q.float(), kc, vc, tables, lens)


def test_sizes_that_are_wrong_are_still_refused():
    q, kc, vc, tables, lens = unused_batch(2, 4, 2, 64, "bf16")
    with pytest.raises((ValueError, _native.EntmaxAttnError)):
        ea.entmax_attn_decode(q, kc, vc, tables, lens, 1.5, max_len=-1)
    with pytest.raises((ValueError, _native.EntmaxAttnError)):
        ea.entmax_attn_decode(q[:, :3], kc, vc, tables, lens, 1.5, max_len=0)
    with pytest.raises((ValueError, _native.EntmaxAttnError)):
        ea.entmax_attn_decode(q, kc, vc, tables, lens, 0.5, max_len=0)
    with pytest.raises(ValueError):
        ea.alloc_decode_workspace(q, kc, -1)
    with pytest.raises((ValueError, _native.EntmaxAttnError)):
        ea.page_tables(lens, lens, lens, lens[:1], tables, 16, -1)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("B", [4, 600])
def test_tables_with_token_counts_that_add_up_past_2_31(B, padded):
    """Huge counts do not fit their table rows; cu_new stops at 2^31 - 1, and no request behind that
    is served (packed), none with a huge count either way."""
    big = (1 << 31) - 1
    new = np.tile([3, big, 7, 5], B // 4)
    if padded:
        new[2] = big
    lens = np.tile([0, 2, 30, 1], B // 4)
    tables = i32(np.full((B, 5), -1))
    free = list(range(4 * B))
    at = np.minimum(np.concatenate([[0], np.cumsum(new)]), big)
    got = ea.page_tables(i32(lens), i32(new), i32(free), i32([0]), tables, 16, 20, padded)
    assert np.array_equal(got[2].cpu().numpy(), at)
    serve = (new < big) & (at[1:] < big) & (padded | (at[1:] <= 20))
    assert serve.any()
    assert np.array_equal(got[1].cpu().numpy(), np.where(serve, lens + new, lens))
    slots = got[0].cpu().numpy()
    assert (slots >= 0).sum() == new[serve].sum()
    assert np.all((tables.cpu().numpy() >= 0).any(1) <= serve)
    if not padded:
        assert (slots[:3] >= 0).all() and (slots[3:] == -1).all()


@pytest.mark.parametrize("raw", [False, True])
def test_the_default_stream_by_its_handle(raw):
    """Handle 0 is the default stream, also while another one is current: the calls see what was
    queued there before them, and what is queued there next sees their results."""
    q, kc, vc, tables, lens = unused_batch(2, 4, 2, 64, "bf16")
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0
    stream = 0 if raw else default
    k = torch.randn(2, 5, 64).bfloat16().cuda()
    new, free, start, table = i32([3, 2]), i32([3, 2, 1]), i32([0]), i32([[0, -1, -1], [1, -1, -1]])
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        with torch.cuda.stream(default):
            torch.cuda._sleep(20_000_000)  # about 10 ms
            tables.copy_(table)
            lens.fill_(1)
        slots, n, _, _ = ea.page_tables(lens, new, free, start, tables, 16, 5, stream=stream)
        ea.paged_append(k, k, kc, vc, slots, stream=stream)
        out, tau = ea.entmax_attn_decode(q, kc, vc, tables, n, 1.5, stream=stream)
        with torch.cuda.stream(default):
            seen = [x.clone() for x in (n, slots, kc, tau)]
    torch.cuda.synchronize()
    assert seen[0].tolist() == [4, 3]
    assert seen[1].tolist() == [1, 2, 3, 17, 18]
    assert torch.equal(seen[2][0, :, 1:4], k[:, :3]) and torch.equal(seen[2][1, :, 1:3], k[:, 3:])
    assert torch.isfinite(seen[3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_of_dimensions_of_one_element_do_not_matter(dtype):
    """k from a projection of its own, v a slice of a fused one: they differ only in the strides of
    the batch, head or token dimension of one element; so do caches of one page or head."""
    d, P = 64, 4
    fused = torch.randn(1, 1, 3 * d).to(DT[dtype]).cuda()
    v = fused[..., 2 * d:].view(1, 1, 1, d)
    k = torch.randn(1, 1, 1, d).to(DT[dtype]).cuda().as_strided((1, 1, 1, d), (8 * d, 1, 7, 1))
    assert k.stride() != v.stride()
    kc = torch.zeros(1, 1, P, d, dtype=DT[dtype], device="cuda")
    vc = torch.zeros(1, P, 1, d, dtype=DT[dtype], device="cuda").transpose(1, 2).as_strided(
        (1, 1, P, d), (3, 5, d, 1))
    assert kc.stride() != vc.stride()
    slots = torch.tensor([2], device="cuda")
    ea.paged_append(k, v, kc, vc, slots)
    assert torch.equal(kc[0, 0, 2], k[0, 0, 0]) and torch.equal(vc[0, 0, 2], v[0, 0, 0])
    ea.paged_append(k[0], v[0], kc, vc, slots)
    q = torch.randn(1, 2, d).to(DT[dtype]).cuda()
    vc[0, 0, 0] = 1.0
    a = ea.entmax_attn_decode(q, kc, vc, i32([[0]]), i32([3]))
    b = ea.entmax_attn_decode(q, kc, vc.clone(memory_format=torch.contiguous_format), i32([[0]]),
                              i32([3]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):  # a difference that matters
        two = torch.zeros(2, 1, P, d, dtype=DT[dtype], device="cuda")
        ea.entmax_attn_decode(q, two, two.expand(2, 1, P, d).as_strided((2, 1, P, d),
                                                                       (d, P * d, d, 1)),
                              i32([[0]]), i32([3]))
