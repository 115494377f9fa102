"""The split decode kernels (scores, then a join) on the cases that batches with a small limit take
to the one-launch kernel.  The kernels are chosen from the sizes and max_len alone, so a wide block
table sends any batch to them; the join is a cluster of 4 blocks per head up to 148 heads, a block up
to 1024, a warp above.  Every call here runs on a workspace full of leftovers, and the prefix sums
that only the split kernels write there are checked, so that a case cannot leave this route
unnoticed."""
import numpy as np
import pytest
import torch

import adaptive_sparse_attention_b200 as ea
from adaptive_sparse_attention_b200 import _native
from oracle import oracle as orc
from oracle import paged
from test_paged_gpu import DT, LENS, Case, i32

pytestmark = pytest.mark.gpu
LIMIT = 200000  # tokens that the block tables address
JOINS = ["4 blocks", "1 block", "warp"]


def repeats(join, heads):
    """How often a batch of `heads` (request, head) pairs is repeated for a form of the join."""
    least, most = {"4 blocks": (1, 148), "1 block": (149, 1024), "warp": (1025, None)}[join]
    n = -(-least // heads)
    if most is not None and n * heads > most:
        pytest.skip("no such batch of these heads")
    return n


def split_run(c, alpha, fill=0x5a, expect=None, **kw):
    """c.run on the split kernels, on a workspace filled with `fill`."""
    ws = ea.alloc_decode_workspace(c.q, c.kc, LIMIT)
    ws.fill_(fill)
    out, tau = c.run(alpha, workspace=ws, max_len=LIMIT, **kw)
    lens = np.asarray(c.lens if expect is None else expect)
    pre = np.concatenate([[0], np.cumsum((lens + 15) // 16)])
    assert np.array_equal(ws[:4 * pre.size].view(torch.int32).cpu().numpy(), pre)
    return out, tau


def case(lens, Hq, Hkv, d, P, *a, **kw):
    return Case(lens, Hq, Hkv, d, P, *a, W_extra=-(-LIMIT // P), **kw)


@pytest.mark.parametrize("join", JOINS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha", [1.25, 1.333, 1.5, 2.0, 3.0])
@pytest.mark.parametrize("d,P,layout", [(64, 16, "heads"), (128, 24, "tokens"), (128, 1, "heads"),
                                        (64, 5, "tokens"), (128, 64, "heads")])
def test_split_matches_oracle(join, dtype, alpha, d, P, layout, oracle):
    n = repeats(join, len(LENS) * 8)
    c = case(LENS * n, 8, 2, d, P, dtype, layout, seed=d + P, fused_q=P == 24)
    c.check(*split_run(c, alpha), alpha, rows=range(len(LENS)))
    assert ea.status() == 0


@pytest.mark.parametrize("join", JOINS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G,Hkv", [(1, 1), (1, 3), (2, 2), (3, 1), (5, 2), (7, 1), (8, 2), (9, 1),
                                   (16, 2), (17, 1), (20, 2), (40, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_split_head_groups(join, dtype, G, Hkv, d, oracle):
    lens = [300, 0, 45, 1]
    n = repeats(join, len(lens) * G * Hkv)
    c = case(lens * n, G * Hkv, Hkv, d, 16, dtype, seed=G)
    c.check(*split_run(c, 1.5), 1.5, rows=range(4))


@pytest.mark.parametrize("join", JOINS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha", [1.1, 1.333, 2.0, 3.0])
@pytest.mark.parametrize("G,Hkv,d,P,layout", [(4, 1, 64, 16, "heads"), (2, 2, 128, 5, "tokens"),
                                              (12, 1, 64, 64, "tokens")])
def test_split_long_requests_with_wide_supports(join, dtype, alpha, G, Hkv, d, P, layout, oracle):
    """Thousands of candidates per head beside few: lists beyond the shared-memory ones, and for the
    warp join heads left to the block."""
    lens = [6000, 3, 0, 2100]
    n = repeats(join, len(lens) * G * Hkv)
    rest = [17, 0, 200, 1] * (n - 1) if join == "warp" else lens * (n - 1)
    c = case(lens + rest, G * Hkv, Hkv, d, P, dtype, layout, seed=31, spikes=0.0)
    out, tau = split_run(c, alpha)
    c.check(out, tau, alpha, rows=[0, 1, 2, 3])
    again = split_run(c, alpha, fill=0xff)
    assert torch.equal(out, again[0]) and torch.equal(tau, again[1])


@pytest.mark.parametrize("join", JOINS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha", [1.333, 1.5, 2.0, 3.0])
def test_split_equal_scores(join, dtype, alpha, oracle):
    """q = 0: p = 1 / n, tau = -n^(1 - alpha).  In units of u = 2^-24 tau's relative error is the
    sum's, at most (n / 32 + 132 + n) u, over beta, and p's the sum's and 4 beta u."""
    lens = [1, 2, 16, 100, 513, 4097, 9000]
    n = repeats(join, len(lens) * 2)
    c = case(lens * n, 2, 1, 64, 16, dtype, seed=5, q_scale=0.0)
    out, tau = split_run(c, alpha)
    u = 2.0 ** -24
    beta = 1.0 / (orc.alpha_as_float32(alpha) - 1.0)
    _, _, v = c.f64()
    for b, m in enumerate(lens):
        rel = (m / 32 + 132 + m + 4 * beta) * u
        want = -float(m) ** (-1.0 / beta)
        assert np.all(np.abs(tau[b].double().cpu().numpy() / want - 1) <= rel / beta + 4 * u), m
        rows = paged.gather(v, c.tables[b], m)[0]
        err = (rel + m * u) * np.abs(rows).mean(axis=0)
        tol = err + (np.abs(rows.mean(axis=0)) + err) * torch.finfo(DT[dtype]).eps / 2
        got = out[b].double().cpu().numpy()
        assert np.all(np.abs(got - rows.mean(axis=0)) <= tol), m


@pytest.mark.parametrize("join", JOINS)
def test_split_nan_and_inf_scores_poison_their_row_only(join, oracle):
    lens = [400, 400, 400]
    n = repeats(join, len(lens) * 4)
    c = case(lens * n, 4, 2, 64, 16, "bf16", seed=10)
    c.kc[int(c.tables[1, 3]), 0, 5] = float("nan")
    page = int(c.tables[2, 1])
    c.kc[page, 1, 5] = float("inf")
    c.kc[page, 1, 5, 1:] = 0.0
    out, tau = split_run(c, 1.5)
    assert torch.isnan(out[1, :2]).all() and torch.isnan(tau[1, :2]).all()
    assert not torch.isnan(out[1, 2:]).any() and not torch.isnan(out[0]).any()
    for h in (2, 3):
        assert torch.isnan(tau[2, h]).item() == (c.q[2, h, 0].item() > 0)
    assert not torch.isnan(tau[2, :2]).any() and not torch.isnan(tau[3:]).any()
    c.check(out, tau, 1.5, rows=[0])
    assert ea.status() == 0


@pytest.mark.parametrize("join", JOINS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_split_bad_page_and_length_are_reported(join, dtype, oracle):
    """The kernels check every page number and length before they use it."""
    lens = [400, 300, 50, 60]
    n = repeats(join, len(lens) * 4)
    c = case(lens * n, 4, 2, 64, 16, dtype, seed=11)
    c.d_tables[1, 4] = c.kc.shape[0]
    c.d_tables[2, 0] = -3
    out, tau = split_run(c, 1.5)
    assert ea.status() == _native.ERANGE and ea.status() == 0
    assert torch.isnan(out[1:3]).all() and torch.isnan(tau[1:3]).all()
    assert not torch.isnan(tau[3:]).any()
    c.check(out, tau, 1.5, rows=[0, 3])
    c.d_tables.copy_(i32(c.tables))
    for bad in (-1, LIMIT + 1):
        c.d_lens[1] = bad
        out, tau = split_run(c, 1.5, expect=[400, 0, 50, 60] + lens * (n - 1))
        assert ea.status() == _native.ERANGE
        assert torch.isnan(out[1]).all() and torch.isnan(tau[1]).all()
        c.check(out, tau, 1.5, rows=[0, 2, 3])


@pytest.mark.parametrize("join", JOINS)
@pytest.mark.parametrize("alpha,G", [(1.333, 4), (1.5, 12), (2.0, 1), (3.0, 4)])
def test_split_same_bits_whatever_the_workspace_holds(join, alpha, G):
    lens = [5000, 0, 777, 2000, 1]
    n = repeats(join, len(lens) * G)
    c = case(lens * n, G, 1, 64, 16, "bf16", seed=8, spikes=0.0)
    first = split_run(c, alpha, fill=0)
    for i in range(10):
        got = split_run(c, alpha, fill=(0, 127, 255, 0x5a)[i % 4])
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_split_unused_batch():
    c = case([0] * 5, 4, 2, 64, 16)
    out, tau = split_run(c, 1.5)
    assert (out == 0).all() and torch.isposinf(tau).all() and ea.status() == 0


@pytest.mark.parametrize("alpha", [1.333, 2.0])
def test_split_on_two_streams_and_in_a_graph(alpha, oracle):
    c = [case([6000, 100, 0], 8, 2, 128, 16, "bf16", seed=s, spikes=0.0) for s in (20, 21)]
    want = [split_run(x, alpha) for x in c]
    ws = [ea.alloc_decode_workspace(x.q, x.kc, LIMIT) for x in c]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in c], [], []
    for x, w in zip(c, ws):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(ea.entmax_attn_decode(x.q, x.kc, x.vc, x.d_tables, x.d_lens, alpha,
                                              max_len=LIMIT, workspace=w))
        graphs.append(gr)
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for x, got, ref in zip(c, outs, want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        x.check(*got, alpha)


@pytest.mark.parametrize("join", JOINS)
def test_split_calls_that_share_a_workspace_end(join):
    """Calls that overlap need a workspace each; with one between them their results are undefined, but
    what they read of it reaches no index beyond their buffers and no barrier, so that both end and
    later calls are right."""
    n = repeats(join, 4 * 8)
    c = [case(lens * n, 8, 2, 64, 16, "bf16", seed=s, spikes=0.0)
         for s, lens in ((20, [6000, 100, 0, 900]), (21, [1, 4000, 9000, 16]))]
    want = [split_run(x, 1.333) for x in c]
    ws = ea.alloc_decode_workspace(c[0].q, c[0].kc, LIMIT)
    streams = [torch.cuda.Stream() for _ in c]
    torch.cuda.synchronize()
    for _ in range(30):
        for x, s in zip(c, streams):
            ea.entmax_attn_decode(x.q, x.kc, x.vc, x.d_tables, x.d_lens, 1.333, max_len=LIMIT,
                                  workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert ea.status() == 0
    for x, ref in zip(c, want):
        got = split_run(x, 1.333)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
