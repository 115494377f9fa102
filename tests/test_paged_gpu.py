"""GPU parity of the paged-cache operators against their fp64 oracle (oracle/paged.py).  The page
tables and the append must agree exactly; the decode within bounds derived from the rounding of its
parts (decode_bounds there)."""
import numpy as np
import pytest
import torch

import adaptive_sparse_attention_b200 as ea
from adaptive_sparse_attention_b200 import _native
from oracle import oracle as orc
from oracle import paged

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


# ------------------------------------------------------------------------------- page tables --

def check_tables(lens, new, free, start, tables, page, n_new, padded, **kw):
    want = paged.page_tables(lens, new, free, start, tables.cpu().numpy(), page, n_new, padded)
    got = ea.page_tables(i32(lens), i32(new), i32(free), i32([start]), tables, page, n_new, padded,
                         **kw)
    for name, a, b in zip(("tables", "slots", "lens", "cu", "next"), want, (tables,) + got):
        assert np.array_equal(a, b.cpu().numpy().reshape(np.shape(a))), name
    return got


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("B", [1, 7, 64, 513, 1000])
def test_tables_match_oracle(B, page, padded):
    rng = np.random.default_rng(B * 100 + page)
    lens = rng.integers(0, 300, size=B)
    new = np.where(rng.random(B) < 0.2, 0, rng.integers(1, 90, size=B))
    new[0] = 1
    W = int((lens + new).max()) // page + 2
    tables = i32(rng.integers(0, 10 ** 6, size=(B, W)))
    need = int(sum(-(-int(a + n) // page) for a, n in zip(lens, new)))
    free = rng.permutation(need + 9)
    n_new = int(new.max()) + 2 if padded else int(new.sum()) + 5
    check_tables(lens, new, free, 3, tables, page, n_new, padded)


@pytest.mark.parametrize("B", [8192])
def test_tables_largest_batch(B):
    rng = np.random.default_rng(0)
    lens, new = rng.integers(0, 100, size=B), rng.integers(0, 3, size=B)
    free = rng.permutation(3 * B)
    check_tables(lens, new, free, 0, i32(np.full((B, 8), -1)), 16, 2, True)
    check_tables(lens, new, free, 0, i32(np.full((B, 8), -1)), 16, int(new.sum()), False)


def test_tables_refuse_what_does_not_fit():
    """Requests with lengths below zero or beyond the table row, tokens beyond the slots, an
    exhausted or absent free list, a start outside it, table entries of -1."""
    full = np.full((6, 4), 77)
    lens, new = [3, 4, 0, 3, -1, 60], [1, 1, 9, 1, 2, 9]
    free = [7, 8, 9, 10]
    for padded, n_new in ((False, 30), (False, 5), (False, 1), (True, 9), (True, 1)):
        for f, start in ((free, 0), (free, 1), (free, 4), (free, 5), (free, -1), ([], 0)):
            check_tables(lens, new, f, start, i32(full), 4, n_new, padded)
    check_tables(lens, new, list(range(30)), 0, i32(full), 4, 30, False)
    check_tables([5, 2], [1, 1], free, 0, i32([[3, -1, 4], [-1, 5, 6]]), 4, 2, False)
    check_tables([0, 0], [0, 0], free, 2, i32([[3, -1], [-1, 5]]), 4, 2, False)


def test_tables_in_a_wider_table_and_given_outputs():
    rng = np.random.default_rng(4)
    wide = i32(rng.integers(0, 99, size=(5, 20)))
    before = wide.clone()
    out = dict(slots=torch.empty(40, dtype=torch.int64, device="cuda"), lens_out=i32([0] * 5),
               cu_new=i32([0] * 6), free_next=i32([0]))
    got = check_tables([0, 9, 3, 8, 1], [8, 8, 8, 8, 8], rng.permutation(50), 2, wide[:, 3:9], 4,
                       40, False, **out)
    assert got[0] is out["slots"] and got[1] is out["lens_out"]
    assert torch.equal(wide[:, :3], before[:, :3]) and torch.equal(wide[:, 9:], before[:, 9:])


# ------------------------------------------------------------------------------------ append --

def new_cache(pages, Hkv, P, d, dtype, layout, seed=0):
    g = torch.Generator().manual_seed(seed)
    shape = (pages, Hkv, P, d) if layout == "heads" else (pages, P, Hkv, d)
    c = torch.randn(shape, generator=g).to(DT[dtype]).cuda()
    return c if layout == "heads" else c.transpose(1, 2)


def bits(t):
    t = t.contiguous().cpu()
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("B,Hkv,T,P", [(1, 1, 1, 1), (0, 2, 7, 5), (3, 2, 5, 16), (64, 8, 1, 64),
                                       (0, 3, 1001, 24), (2, 8, 333, 16)])
def test_append_matches_oracle(dtype, d, layout, B, Hkv, T, P):
    """B = 0 stands for the packed layout.  k and v are slices of a fused projection's output
    (strided heads and tokens); some slots are negative."""
    rng = np.random.default_rng(T)
    N = max(B, 1) * T
    pages = -(-N // P) + 2
    kc, vc = (new_cache(pages, Hkv, P, d, dtype, layout, s) for s in (1, 2))
    slots = rng.permutation(pages * P)[:N]
    slots[rng.random(N) < 0.1] = -1
    fused = torch.randn(max(B, 1), T, 2 * Hkv * d + 8,
                        generator=torch.Generator().manual_seed(3)).to(DT[dtype]).cuda()
    k, v = (fused[..., i * Hkv * d:(i + 1) * Hkv * d].unflatten(-1, (Hkv, d)).transpose(1, 2)
            for i in (0, 1))
    wk, wv = (paged.append(bits(c), bits(x.transpose(0, 1)).reshape(Hkv, N, d), slots)
              for c, x in ((kc, k), (vc, v)))
    if B == 0:
        k, v = k[0], v[0]
    ea.paged_append(k, v, kc, vc, torch.from_numpy(slots).cuda())
    assert np.array_equal(bits(kc), wk) and np.array_equal(bits(vc), wv)
    assert ea.status() == 0


def test_append_skips_and_reports_slots_beyond_the_cache():
    kc, vc = (new_cache(3, 2, 4, 64, "bf16", "heads", s) for s in (1, 2))
    k = torch.randn(2, 4, 64).bfloat16().cuda()
    slots = torch.tensor([5, 12, 1 << 40, -7]).cuda()
    want = paged.append(bits(kc), bits(k), [5, -1, -1, -1])
    ea.paged_append(k, k, kc, vc, slots)
    assert ea.status() == _native.ERANGE and ea.status() == 0
    assert np.array_equal(bits(kc), want)


def test_append_of_nothing():
    kc = new_cache(2, 2, 4, 64, "bf16", "heads")
    none = torch.empty(2, 0, 64, dtype=torch.bfloat16, device="cuda")
    ea.paged_append(none, none, kc, kc.clone(), torch.empty(0, dtype=torch.int64, device="cuda"))


# ------------------------------------------------------------------------------------ decode --

class Case:
    """A batch of requests in scattered pages; what lies outside the requests is NaN."""

    def __init__(self, lens, Hq, Hkv, d, P, dtype="bf16", layout="heads", seed=0, spikes=0.02,
                 q_scale=1.0, fused_q=False, W_extra=0):
        rng = np.random.default_rng(seed)
        nb = [-(-n // P) for n in lens]
        pages = sum(nb) + 2
        ids = rng.permutation(pages)
        W = max(1, max(nb)) + W_extra
        self.tables = np.full((len(lens), W), -1)
        self.kc, self.vc = (new_cache(pages, Hkv, P, d, dtype, layout, seed + s) for s in (1, 2))
        used = torch.zeros(pages, P, dtype=torch.bool)
        at = 0
        for b, n in enumerate(lens):
            self.tables[b, :nb[b]] = ids[at:at + nb[b]]
            j = np.arange(n)
            used[self.tables[b, j // P], j % P] = True
            at += nb[b]
        if spikes:
            hit = torch.from_numpy(rng.random((pages, Hkv, P, 1)) < spikes).cuda()
            self.kc.mul_(torch.where(hit, 4.0, 1.0).to(self.kc.dtype))
        dead = ~used.cuda()[:, None, :, None]
        self.kc.masked_fill_(dead, float("nan"))
        self.vc.masked_fill_(dead, float("nan"))
        B = len(lens)
        q = torch.randn(B, (Hq + 2 * Hkv) * d if fused_q else Hq * d,
                        generator=torch.Generator().manual_seed(seed)) * q_scale
        self.q = q.to(DT[dtype]).cuda()[:, :Hq * d].view(B, Hq, d)
        self.lens, self.dtype = list(lens), dtype
        self.d_tables, self.d_lens = i32(self.tables), i32(lens)

    def run(self, alpha, n_iter=10, **kw):
        out, tau = ea.entmax_attn_decode(self.q, self.kc, self.vc, self.d_tables, self.d_lens,
                                         alpha, n_iter, **kw)
        torch.cuda.synchronize()
        return out, tau

    def f64(self):
        return (t.float().cpu().numpy().astype(np.float64) for t in (self.q, self.kc, self.vc))

    def check(self, out, tau, alpha, rows=None):
        rows = range(len(self.lens)) if rows is None else rows
        lens = [n if b in rows else 0 for b, n in enumerate(self.lens)]
        a32 = orc.alpha_as_float32(alpha)
        q, k, v = self.f64()
        o, t = paged.decode(q, k, v, self.tables, lens, a32)
        eps = torch.finfo(DT[self.dtype]).eps
        bo, bt = paged.decode_bounds(q, k, v, self.tables, lens, a32, t, eps)
        got_o, got_t = out.float().cpu().numpy().astype(float).reshape(o.shape), tau.cpu().numpy()
        got_t = got_t.astype(float).reshape(t.shape)
        for b in rows:
            if self.lens[b] == 0:
                assert (got_o[b] == 0).all() and np.isposinf(got_t[b]).all()
                continue
            assert np.all(np.abs(got_t[b] - t[b]) <= bt[b]), (b, np.abs(got_t[b] - t[b]).max())
            assert np.all(np.abs(got_o[b] - o[b]) <= bo[b]), \
                (b, float((np.abs(got_o[b] - o[b]) / bo[b]).max()))


LENS = [0, 1, 2, 15, 16, 17, 33, 0, 127, 128, 129, 1000, 700, 0]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha,n_iter", [(1.333, 10), (1.5, 10), (2.0, 10), (3.0, 40),
                                          (1.25, 20)])
@pytest.mark.parametrize("d,P,layout", [(64, 16, "heads"), (128, 24, "tokens"), (128, 1, "heads"),
                                        (64, 5, "tokens"), (128, 64, "heads")])
def test_decode_matches_oracle(dtype, alpha, n_iter, d, P, layout, oracle):
    c = Case(LENS, 8, 2, d, P, dtype, layout, seed=d + P, fused_q=P == 24)
    c.check(*c.run(alpha, n_iter), alpha)
    assert ea.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G,Hkv", [(1, 1), (1, 3), (2, 2), (3, 1), (5, 2), (7, 1), (8, 2), (9, 1),
                                   (16, 2), (17, 1), (20, 2), (40, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_head_groups(dtype, G, Hkv, d, oracle):
    c = Case([300, 0, 45, 1], G * Hkv, Hkv, d, 16, dtype, seed=G, W_extra=3)
    c.check(*c.run(1.5), 1.5)


@pytest.mark.parametrize("alpha", [1.333, 1.5, 2.0])
@pytest.mark.parametrize("lens", [[20000], [3, 30000, 0, 41, 5000], [9000] * 3])
def test_decode_long_and_ragged(alpha, lens, oracle):
    for spikes, q_scale in ((0.02, 1.0), (0.0, 1.0), (0.0, 0.2)):
        c = Case(lens, 4, 1, 128, 64, "bf16", seed=7, spikes=spikes, q_scale=q_scale)
        c.check(*c.run(alpha), alpha)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha", [1.05, 1.1])
@pytest.mark.parametrize("lens,Hq,Hkv", [([3000, 7, 1200], 4, 2), ([9000] * 2, 4, 1),
                                         ([2500] * 12, 32, 16)])
def test_decode_supports_as_wide_as_the_cache(dtype, alpha, lens, Hq, Hkv, oracle):
    """alpha near 1: every key lies within 1 of the largest score (in z units) and most have p > 0,
    so the candidates overflow the shared-memory lists; the cases take the cluster kernel and both
    block joins of the split kernels."""
    c = Case(lens, Hq, Hkv, 64, 16, dtype, seed=16, spikes=0.0)
    out, tau = c.run(alpha)
    c.check(out, tau, alpha, rows=range(min(3, len(lens))))


@pytest.mark.parametrize("alpha,spikes", [(1.333, 0.0), (1.5, 0.02), (2.0, 0.0), (1.1, 0.0)])
def test_decode_more_heads_than_blocks(alpha, spikes, oracle):
    """Above 1024 heads the join takes a warp per head; some with more candidates than a warp is
    given (those of the long requests), some with none."""
    lens = ([5, 3000, 60, 0, 200, 1, 90, 1500, 17, 16] * 4)
    c = Case(lens, 32, 8, 64, 16, "bf16", seed=17, spikes=spikes)
    out, tau = c.run(alpha)
    c.check(out, tau, alpha, rows=[0, 1, 3, 7, 12, 29, 39])
    again = c.run(alpha)
    assert torch.equal(out, again[0]) and torch.equal(tau, again[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha,n_iter", [(1.333, 10), (1.5, 10), (2.0, 10), (3.0, 40)])
def test_decode_equal_scores(dtype, alpha, n_iter, oracle):
    """q = 0: every key ties, p = 1/n, tau = -n^(1 - alpha); supports as wide as the cache."""
    lens = [1, 2, 16, 100, 513, 4097, 9000]
    c = Case(lens, 2, 1, 64, 16, dtype, seed=5, q_scale=0.0)
    out, tau = c.run(alpha, n_iter)
    a32 = orc.alpha_as_float32(alpha)
    want = np.array([-float(n) ** (1.0 - a32) for n in lens])
    got = tau.cpu().numpy().astype(float)
    # relative: p depends on tau^beta
    assert np.all(np.abs(got / want[:, None] - 1.0) <= 1e-5), (got, want)
    _, _, v = c.f64()
    for b, n in enumerate(lens):
        mean = paged.gather(v, c.tables[b], n)[0].mean(axis=0)
        eps = torch.finfo(DT[dtype]).eps
        # p off by beta 1e-5 relative, the sum by n 2^-24 of sum |v| / n, o's rounding
        tol = (1e-5 / (a32 - 1.0) + n * 2.0 ** -24 + 1e-6) * 4.0 + np.abs(mean) * eps / 2
        assert np.all(np.abs(out[b].float().cpu().numpy() - mean) <= tol), n


def test_decode_half_the_keys_tie_far_above_the_rest(oracle):
    c = Case([4000, 1500], 4, 2, 64, 16, "fp32", seed=6, spikes=0.0)
    c.kc.copy_(torch.where(torch.isnan(c.kc), c.kc, torch.zeros_like(c.kc)))
    far = torch.rand(c.kc.shape[:3], device="cuda")[..., None] < 0.5
    c.kc.copy_(torch.where(far & ~torch.isnan(c.kc), torch.full_like(c.kc, 0.5), c.kc))
    for alpha in (1.5, 2.0):
        c.check(*c.run(alpha), alpha)


def test_decode_same_bits_again_and_dirty_workspace(oracle):
    c = Case([5000, 0, 777, 12000, 1], 8, 2, 128, 16, "bf16", seed=8, spikes=0.0)
    ws = ea.alloc_decode_workspace(c.q, c.kc, 12000)
    ws.fill_(0)
    a = c.run(1.333, workspace=ws, max_len=12000)
    for fill in (255, 127):
        ws.fill_(fill)
        b = c.run(1.333, workspace=ws, max_len=12000)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    b = c.run(1.333)  # its own workspace, max_len from the table
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("lens,Hq,Hkv,alpha,spikes", [
    ([1000], 32, 8, 1.5, 0.02), ([4096] * 4, 8, 2, 1.333, 0.0), ([2000, 900, 1500], 16, 1, 2.0, 0.0),
    ([700] * 40, 8, 4, 1.333, 0.0), ([3000] * 16, 8, 8, 1.5, 0.0), ([20000, 8000], 8, 2, 1.333, 0.0)])
def test_decode_same_bits_many_times(lens, Hq, Hkv, alpha, spikes):
    """The warps of a cluster share their running maxima, so which candidates they store depends on
    the timing; the results must not."""
    c = Case(lens, Hq, Hkv, 64, 16, "bf16", seed=15, spikes=spikes)
    ws = ea.alloc_decode_workspace(c.q, c.kc, max(lens))
    first = None
    for _ in range(40):
        got = ea.entmax_attn_decode(c.q, c.kc, c.vc, c.d_tables, c.d_lens, alpha,
                                    max_len=max(lens), workspace=ws)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_decode_layout_variants_agree():
    """[B, Hq, 1, d], given outputs, a table that is a slice of a wider one."""
    c = Case([500, 20], 4, 2, 64, 16, "bf16", seed=9)
    a = c.run(1.5)
    out, tau = torch.empty_like(c.q).unsqueeze(2), torch.empty(2, 4, 1, device="cuda")
    wide = torch.full((2, 50), -5, dtype=torch.int32, device="cuda")
    wide[:, 7:7 + c.d_tables.shape[1]] = c.d_tables
    got = ea.entmax_attn_decode(c.q.unsqueeze(2), c.kc, c.vc, wide[:, 7:7 + c.d_tables.shape[1]],
                                c.d_lens, 1.5, out=out, tau=tau)
    assert got[0] is out and got[1] is tau
    assert torch.equal(out[:, :, 0], a[0]) and torch.equal(tau[:, :, 0], a[1])


def test_decode_nan_and_inf_scores_poison_their_row_only(oracle):
    c = Case([400, 400, 400], 4, 2, 64, 16, "bf16", seed=10)
    page = int(c.tables[1, 3])
    c.kc[page, 0, 5] = float("nan")
    page2 = int(c.tables[2, 1])
    c.kc[page2, 1, 5] = float("inf")
    c.kc[page2, 1, 5, 1:] = 0.0
    out, tau = c.run(1.5)
    assert torch.isnan(out[1, :2]).all() and torch.isnan(tau[1, :2]).all()
    assert not torch.isnan(out[1, 2:]).any() and not torch.isnan(out[0]).any()
    # inf x q: +inf for the heads whose first element is positive, -inf (p = 0) for the others
    for h in (2, 3):
        assert torch.isnan(tau[2, h]).item() == (c.q[2, h, 0].item() > 0)
    assert not torch.isnan(tau[2, :2]).any()
    c.check(out, tau, 1.5, rows=[0])
    assert ea.status() == 0


def test_decode_bad_page_and_length_are_reported(oracle):
    """The kernels check every page number and length before they use it."""
    c = Case([400, 300, 50, 60], 4, 2, 64, 16, "bf16", seed=11)
    c.d_tables[1, 4] = c.kc.shape[0]
    c.d_tables[2, 0] = -3
    out, tau = c.run(1.5)
    assert ea.status() == _native.ERANGE and ea.status() == 0
    assert torch.isnan(out[1:3]).all() and torch.isnan(tau[1:3]).all()
    c.check(out, tau, 1.5, rows=[0, 3])
    c.d_tables.copy_(i32(c.tables))
    for bad in (-1, 401):
        c.d_lens.copy_(i32([400, bad, 50, 60]))
        out, tau = c.run(1.5, max_len=400)
        assert ea.status() == _native.ERANGE
        assert torch.isnan(out[1]).all() and torch.isnan(tau[1]).all()
        c.check(out, tau, 1.5, rows=[0, 2, 3])


def test_decode_offsets_beyond_32_bits(oracle):
    """A cache of more than 2^32 bytes and 2^31 elements; the pages in use lie at its end."""
    Hkv, P, d = 8, 128, 128
    pages = (1 << 31) // (Hkv * P * d) + 40
    kc = torch.empty(pages, Hkv, P, d, dtype=torch.bfloat16, device="cuda")
    small = Case([3000, 1000], 8, Hkv, d, P, "bf16", seed=12)
    n = small.kc.shape[0]
    kc[-n:] = small.kc
    vc = torch.empty_like(kc)
    vc[-n:] = small.vc
    a = small.run(1.5)
    tables = torch.where(small.d_tables >= 0, small.d_tables + (pages - n), small.d_tables)
    b = ea.entmax_attn_decode(small.q, kc, vc, tables, small.d_lens, 1.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    new = torch.randn(Hkv, 3, d, device="cuda").bfloat16()
    slots = torch.tensor([pages * P - 1, (pages - 1) * P, pages * P - 7]).cuda()
    ea.paged_append(new, new, kc, vc, slots)
    got = torch.stack([kc[-1, :, -1], kc[-1, :, 0], kc[-1, :, -7]], 1)
    assert torch.equal(got, new) and ea.status() == 0


def test_largest_batch(oracle):
    rng = np.random.default_rng(13)
    lens = rng.integers(0, 40, size=8192).tolist()
    c = Case(lens, 2, 1, 64, 16, "bf16", seed=13)
    out, tau = c.run(1.5)
    c.check(out, tau, 1.5, rows=[0, 1, 2, 500, 4095, 4096, 8000, 8190, 8191])
    empty = torch.tensor(lens).cuda() == 0
    assert (out[empty] == 0).all() and torch.isinf(tau[empty]).all()
    assert torch.isfinite(tau[~empty]).all()


# ---------------------------------------------------------------------- streams, graphs, steps --

def test_other_streams_with_their_own_workspaces(oracle):
    c = [Case([6000, 100, 0], 8, 2, 128, 16, "bf16", seed=s) for s in (20, 21)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in c]
    got = []
    for _ in range(3):
        got = [ea.entmax_attn_decode(x.q, x.kc, x.vc, x.d_tables, x.d_lens, 1.5, stream=s)
               for x, s in zip(c, streams)]
    raw = ea.entmax_attn_decode(c[0].q, c[0].kc, c[0].vc, c[0].d_tables, c[0].d_lens, 1.5,
                                stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    for x, (out, tau) in zip(c, got):
        x.check(out, tau, 1.5)
    assert torch.equal(raw[0], got[0][0])


def test_graph_replays_as_the_requests_grow(oracle):
    """A captured step (tables, append, decode), replayed: the lengths, tables and free list live
    on the device, so every replay appends one token per request and attends to it.  Two graphs
    over one workspace, replayed in turn."""
    B, Hq, Hkv, d, P, W = 5, 4, 2, 64, 16, 6
    rng = np.random.default_rng(30)
    kc, vc = (new_cache(40, Hkv, P, d, "bf16", "heads", s) for s in (1, 2))
    free = i32(rng.permutation(40))
    start = i32([0])
    tables = i32(np.full((B, W), -1))
    lens = i32([0] * B)
    new = i32([30, 15, 16, 1, 0])
    slots, l2, _, s2 = ea.page_tables(lens, new, free, start, tables, P, 62)
    k0, v0 = (torch.randn(Hkv, 62, d, device="cuda").bfloat16() for _ in range(2))
    ea.paged_append(k0, v0, kc, vc, slots)
    lens.copy_(l2)
    start.copy_(s2)
    one = i32([1] * B)
    k, v, q = (torch.zeros(B, h, 1, d, device="cuda", dtype=torch.bfloat16)
               for h in (Hkv, Hkv, Hq))
    ws = ea.alloc_decode_workspace(q, kc, W * P)
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first calls outside the capture
        ea.entmax_attn_decode(q, kc, vc, tables, lens, 1.5, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for alpha in (1.5, 2.0):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            slots, l2, _, s2 = ea.page_tables(lens, one, free, start, tables, P, 1, padded=True)
            ea.paged_append(k, v, kc, vc, slots)
            outs.append(ea.entmax_attn_decode(q, kc, vc, tables, l2, alpha, workspace=ws))
            lens.copy_(l2)
            start.copy_(s2)
        graphs.append(gr)
    n = [30, 15, 16, 1, 0]
    for step in range(20):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(step)))
        which = step % 2
        graphs[which].replay()
        torch.cuda.synchronize()
        n = [x + 1 for x in n]
        assert lens.tolist() == n
        c = Case.__new__(Case)
        c.q, c.kc, c.vc, c.lens, c.dtype = q[:, :, 0], kc, vc, n, "bf16"
        c.tables = tables.cpu().numpy()
        out, tau = outs[which]
        c.check(out[:, :, 0], tau[:, :, 0], (1.5, 2.0)[which])
        slot = c.tables[np.arange(B), (np.array(n) - 1) // P], (np.array(n) - 1) % P
        assert torch.equal(kc[torch.from_numpy(slot[0]).cuda(), :,
                              torch.from_numpy(slot[1]).cuda()], k[:, :, 0])
    assert ea.status() == 0


def test_prefill_then_decode_agrees_with_the_forward_pass(oracle):
    """The packed forward pass over whole sequences against prefill + append of all but the last
    token, then one decoding step: the last rows agree."""
    from adaptive_sparse_attention_b200.workloads import random_case
    lens = (200, 1, 777, 64)
    w, (q, k, v, cu) = random_case(B=None, Hq=8, Hkv=2, T=None, d=128, alpha=1.5, seqlens=lens,
                                   spike_frac=0.02, spike_scale=4.0, seed=3)
    q, k, v, cu = (x.cuda() for x in (q, k, v, cu))
    want, wtau, _ = ea.entmax_attn_fwd(q, k, v, 1.5, 10, True, cu)
    B, P, W = len(lens), 16, 50
    kc, vc = (torch.full((70, 2, P, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    free, start, tables = i32(np.random.default_rng(0).permutation(70)), i32([0]), \
        i32(np.full((B, W), -1))
    first = [n - 1 for n in lens]
    keep = torch.cat([torch.arange(int(cu[b]), int(cu[b]) + n) for b, n in enumerate(first)])
    slots, n1, cu1, start = ea.page_tables(i32([0] * B), i32(first), free, start, tables, P,
                                           sum(first))
    assert cu1.tolist() == np.concatenate([[0], np.cumsum(first)]).tolist()
    ea.paged_append(k[:, keep], v[:, keep], kc, vc, slots)
    last = (cu[1:] - 1).long()
    slots, n2, _, _ = ea.page_tables(n1, i32([1] * B), free, start, tables, P, 1, padded=True)
    kl, vl, ql = (x[:, last].transpose(0, 1).unsqueeze(2).contiguous() for x in (k, v, q))
    ea.paged_append(kl, vl, kc, vc, slots)
    out, tau = ea.entmax_attn_decode(ql, kc, vc, tables, n2, 1.5)
    assert n2.tolist() == list(lens)
    o = want[:, last].transpose(0, 1).float()
    # both within their bars of the exact value: 2e-2 + 2^-9 |o| for the forward pass, less for
    # the decode; tau within 1e-4 max(1, |tau|)
    assert torch.all((out[:, :, 0].float() - o).abs() <= 2 * (2e-2 + 2.0 ** -8 * o.abs()))
    t = wtau[:, last].transpose(0, 1)
    assert torch.all((tau[:, :, 0] - t).abs() <= 2e-4 * t.abs().clamp(min=1.0))
    assert ea.status() == 0


def test_binding_refusals():
    c = Case([40, 20], 4, 2, 64, 16, "bf16", seed=14)
    with pytest.raises(ValueError):
        ea.entmax_attn_decode(c.q.float(), c.kc, c.vc, c.d_tables, c.d_lens)
    with pytest.raises(ValueError):
        ea.entmax_attn_decode(c.q, c.kc, c.vc.transpose(1, 2), c.d_tables, c.d_lens)
    with pytest.raises(ValueError):
        ea.entmax_attn_decode(c.q, c.kc, c.vc, c.d_tables.long(), c.d_lens)
    with pytest.raises(ValueError):
        ea.entmax_attn_decode(c.q, c.kc, c.vc, c.d_tables, c.d_lens[:1])
    with pytest.raises(ValueError):
        ea.entmax_attn_decode(c.q, c.kc, c.vc, c.d_tables, c.d_lens.cpu())
    with pytest.raises(_native_error()):
        ea.entmax_attn_decode(c.q, c.kc, c.vc, c.d_tables, c.d_lens, max_len=10 ** 6)
    with pytest.raises(_native_error()):
        ea.entmax_attn_decode(c.q, c.kc, c.vc, c.d_tables, c.d_lens,
                              workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(_native_error()):
        ea.entmax_attn_decode(c.q, c.kc, c.vc, c.d_tables[:1].expand(2, -1), c.d_lens)
    with pytest.raises(ValueError):
        ea.paged_append(c.q, c.q, c.kc, c.vc, torch.zeros(2, dtype=torch.int64).cuda())
    with pytest.raises(_native_error()):
        ea.page_tables(c.d_lens, c.d_lens, c.d_lens, c.d_lens[:1], c.d_tables, 16, 8,
                       lens_out=c.d_lens)


def _native_error():
    return _native.EntmaxAttnError
