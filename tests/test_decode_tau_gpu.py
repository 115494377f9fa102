"""One-token attention where tau lies far from 0 or close to the largest score: p = (z - tau)^beta
is made of differences, so they must be resolved whatever the scores' own size."""
import numpy as np
import pytest
import torch

import adaptive_sparse_attention_b200 as ea
from oracle import oracle as orc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24


def tied(n, score, alpha, dtype, d=64, others=()):
    """One request of one head whose n keys all have z = score up to the rounding of q, in pages of
    16, values above 0; `others`: scores of further keys.  Returns (q, kc, vc, table, lens, z)."""
    a32 = orc.alpha_as_float32(alpha)
    c = (a32 - 1.0) / np.sqrt(d)
    total = n + len(others)
    pages = -(-total // 16)
    g = torch.Generator().manual_seed(n)
    q = torch.zeros(1, 1, d, dtype=DT[dtype])
    k = torch.zeros(pages * 16, d, dtype=DT[dtype])
    q[0, 0, 0], k[:, 0] = 1.0, score / c
    for i, x in enumerate(others):
        k[n + i, 0] = x / c
    v = torch.randn(pages * 16, d, generator=g).abs().to(DT[dtype])
    kc, vc = (x.view(pages, 1, 16, d).cuda() for x in (k, v))
    table = torch.arange(pages, dtype=torch.int32).view(1, -1).cuda()
    lens = torch.tensor([total], dtype=torch.int32).cuda()
    return q.cuda(), kc, vc, table, lens, c * k[:total, 0].double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha", [1.333, 1.5, 2.0, 3.0])
@pytest.mark.parametrize("n", [2, 300, 9000, 100000])
@pytest.mark.parametrize("score", [8.0, 16.0, 30.0, -60.0, 1e5, 2.0 ** 23 + 1, 1e9])
def test_tied_scores_far_from_zero(dtype, alpha, n, score):
    """p = 1 / n whatever the scores, so o is the mean of v.  In units of u = 2^-24: the sums that
    tau is solved from add at most n / 32 + 64 terms after one another, the power is good to 64 u,
    tau settles to 4 u of m - tau; so p is off by (n / 32 + 132 + 4 beta) u relative and the sum of
    p v by n u more, then o is rounded."""
    q, kc, vc, table, lens, z = tied(n, score, alpha, dtype)
    out, tau = ea.entmax_attn_decode(q, kc, vc, table, lens, alpha, 60)
    beta = 1.0 / (orc.alpha_as_float32(alpha) - 1.0)
    mean = vc.double().view(-1, 64)[:n].mean(0).cpu().numpy()
    err = (n / 32 + 132 + 4 * beta + n) * U * mean
    tol = err + (mean + err) * torch.finfo(DT[dtype]).eps / 2
    got = out[0, 0].double().cpu().numpy()
    assert np.all(np.abs(got - mean) <= tol), float(np.abs(got / mean - 1).max())
    # tau = z - n^(1 - alpha); z = c q k rounds twice, tau once more
    want = z[0] - float(n) ** (-1.0 / beta)
    rel = (n / 32 + 132 + 4 * beta + n) * U / beta
    assert abs(float(tau) - want) <= 3 * U * abs(z[0]) + rel * float(n) ** (-1.0 / beta) + \
        U * abs(want)


@pytest.mark.parametrize("alpha", [1.5, 2.0])
def test_scores_beyond_the_integers_of_fp32(alpha):
    """Two keys tie above 2^23, others lie several units below: p = 1/2, 1/2, 0, ..."""
    top = 2.0 ** 24 + 64
    q, kc, vc, table, lens, z = tied(2, top, alpha, "fp32", others=[top - 16, -top, 0.0])
    assert z[0] - z[2] > 4  # what the rounding of k leaves of it
    out, tau = ea.entmax_attn_decode(q, kc, vc, table, lens, alpha)
    v = vc.double().view(-1, 64)
    want = 0.5 * (v[0] + v[1])
    assert torch.all((out[0, 0].double() - want).abs() <= 200 * U * want)
    assert abs(float(tau) - z[0]) <= 4 * U * top


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha", [1.333, 1.5, 2.0])
@pytest.mark.parametrize("max_len", [None, 200000])
def test_a_common_shift_of_the_scores_changes_nothing(dtype, alpha, max_len):
    """Adding the same exactly representable number to every score leaves p alone.  Scores are
    multiples of 2^-10 below 8 in size, shifted by 0 or 64 (24 bits hold both), c a power of two
    times alpha - 1, applied by one rounding; so z - max differs by the roundings of c q k alone:
    2 u 72 absolute for x = z - tau, hence |dp| <= beta p^(1 - 1/beta) 4 u 72 (x <= 1)."""
    n, d, W = 3000, 64, -(-(max_len or 3008) // 16)
    rng = np.random.default_rng(3)
    a32 = orc.alpha_as_float32(alpha)
    raw = np.round(rng.uniform(-4, 4, n) * 1024) / 1024 * 8  # c = (alpha - 1) / 8
    v = torch.from_numpy(rng.uniform(0.5, 1.5, (1, 1, 3008, d))).to(DT[dtype])
    outs = []
    for shift in (0.0, 512.0):
        k = torch.zeros(188, 1, 16, d)
        kv = k.view(-1, d)
        kv[:n, 0] = torch.from_numpy(raw).float()
        kv[:n, 1] = shift
        # bf16 holds 8 bits: the score in three pieces, q = 1 for each
        if dtype == "bf16":
            hi = kv[:, 0].bfloat16().float()
            mid = (kv[:, 0] - hi).bfloat16().float()
            kv[:, 2], kv[:, 3], kv[:, 0] = mid, kv[:, 0] - hi - mid, hi
        q = torch.zeros(1, 1, d)
        q[..., :4] = 1.0
        kc = k.to(DT[dtype]).cuda()
        assert torch.equal(kc.float().cpu(), k)
        table = torch.full((1, W), -1, dtype=torch.int32)
        table[0, :188] = torch.arange(188)
        outs.append(ea.entmax_attn_decode(q.to(DT[dtype]).cuda(), kc,
                                          v.view(188, 1, 16, d).cuda(), table.cuda(),
                                          torch.tensor([n], dtype=torch.int32).cuda(), alpha,
                                          max_len=max_len))
    z = (a32 - 1.0) / 8 * raw
    p, _ = orc.entmax_vec(z, a32)
    beta = 1.0 / (a32 - 1.0)
    dx = 4 * U * 72
    dp = beta * (p ** (1 / beta) + dx) ** (beta - 1) * dx * (p > 0) + dx ** beta * (
        np.abs(z - z[p > 0].min()) <= dx) + 132 * U * p
    vv = v.double().numpy().reshape(-1, d)[:n]
    want = p @ vv
    err = 2 * dp.sum() * 1.5 + n * U * want.max()
    tol = err + (want + err) * torch.finfo(DT[dtype]).eps / 2
    for out, _ in outs:
        assert np.all(np.abs(out[0, 0].double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("alpha", [2.1, 3.0, 4.0, 8.0])
@pytest.mark.parametrize("n,heads,max_len", [(1, 4, None), (2, 4, None), (50, 8, None),
                                             (1000, 8, None), (20000, 4, None), (20000, 160, None),
                                             (1000, 8, 200000)])
@pytest.mark.parametrize("spread", [0.0, 0.01, 0.3, 1.0, 5.0])
def test_alpha_above_two_settles_by_itself(dtype, alpha, n, heads, max_len, spread, oracle):
    """For alpha > 2 the sum of the p has a cusp at every score (p rises with an infinite slope), on
    which steps by derivatives stall or stop short of the root.  The default n_iter; the scores'
    standard deviation is `spread` (every score ties at 0).  Bounds: oracle.paged.decode_bounds."""
    from oracle import paged
    d, P = 64, 16
    a32 = orc.alpha_as_float32(alpha)
    g = torch.Generator().manual_seed(n + heads)
    pages = -(-n // P)
    W = -(-(max_len or n) // P)
    kc, vc = (torch.randn(pages, 1, P, d, generator=g).to(DT[dtype]) for _ in range(2))
    q = (torch.randn(1, heads, d, generator=g) * (spread / (a32 - 1.0))).to(DT[dtype])
    table = np.full((1, W), -1)
    table[0, :pages] = np.arange(pages)
    out, tau = ea.entmax_attn_decode(
        q.cuda(), kc.cuda(), vc.cuda(), torch.from_numpy(table).int().cuda(),
        torch.tensor([n], dtype=torch.int32).cuda(), alpha, max_len=max_len)
    rows = slice(0, 8)  # of the heads: the oracle's time
    qd, kd, vd = (x.double().numpy() for x in (q[:, rows], kc, vc))
    o, t = paged.decode(qd, kd, vd, table, [n], a32)
    bo, bt = paged.decode_bounds(qd, kd, vd, table, [n], a32, t, torch.finfo(DT[dtype]).eps)
    assert np.all(np.abs(tau[:, rows].double().cpu().numpy() - t) <= bt)
    assert np.all(np.abs(out[:, rows].double().cpu().numpy() - o) <= bo)
