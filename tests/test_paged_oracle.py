"""The paged cache's oracle (CPU): page tables against their invariants, the append against a
dictionary, and the one-token attention against the forward oracle's last row."""
import numpy as np
import pytest

from oracle import oracle as orc
from oracle import paged


@pytest.mark.parametrize("page", [1, 5, 16])
@pytest.mark.parametrize("padded", [False, True])
def test_tables_invariants_over_steps(page, padded):
    """Several steps in a row: every token of every request keeps one slot of its own, the tables
    hold each page once, and the free list is used in order without gaps."""
    rng = np.random.default_rng(page)
    B, W = 7, 12
    free = rng.permutation(B * W).tolist()
    tables, lens, start = np.full((B, W), -1), np.zeros(B, dtype=int), 0
    owner = {}
    for _ in range(6):
        new = rng.integers(0, 2 * page + 2, size=B)
        new = np.minimum(new, W * page - lens)
        n_new = int(new.max()) if padded else int(new.sum()) + 3
        if n_new == 0:
            continue
        tables, slots, out, cu, nxt = paged.page_tables(lens, new, free, start, tables, page,
                                                        n_new, padded)
        assert np.array_equal(out, lens + new)
        assert nxt - start == sum(-(-int(o) // page) + (int(x) // -page)
                                  for o, x in zip(out, lens))
        for b in range(B):
            for t in range(int(new[b])):
                s = int(slots[b, t] if padded else slots[cu[b] + t])
                assert s not in owner
                owner[s] = (b, int(lens[b]) + t)
                pos = int(lens[b]) + t
                assert tables[b, pos // page] * page + pos % page == s
        assert (slots >= 0).sum() == new.sum()
        lens, start = out, nxt
    used = tables[tables >= 0]
    assert sorted(used.tolist()) == sorted(free[:start])


def test_tables_out_of_pages_serves_in_order():
    t, slots, out, cu, nxt = paged.page_tables([3, 4, 0, 3], [1, 1, 9, 1], [7, 8, 9], 1,
                                               np.full((4, 4), 5), 4, 12)
    # request 0 needs no page, 1 takes page 8, 2 needs three and has one left, 3 needs none
    assert out.tolist() == [4, 5, 0, 4] and nxt == 2
    assert cu.tolist() == [0, 1, 2, 11, 12]
    assert slots.tolist() == [23, 32] + [-1] * 9 + [23]
    assert t[1].tolist() == [5, 8, 5, 5] and (t[2] == 5).all()


def test_append_writes_its_slots_only():
    rng = np.random.default_rng(1)
    cache = rng.standard_normal((5, 2, 3, 4))
    rows = rng.standard_normal((2, 4, 4))
    out = paged.append(cache, rows, [14, -1, 3, 99])
    assert np.array_equal(out[4, :, 2], rows[:, 0]) and np.array_equal(out[1, :, 0], rows[:, 2])
    same = np.ones((5, 3), dtype=bool)
    same[4, 2] = same[1, 0] = False
    assert np.array_equal(out.transpose(0, 2, 1, 3)[same], cache.transpose(0, 2, 1, 3)[same])


@pytest.mark.parametrize("alpha", [1.333, 1.5, 2.0, 3.0])
def test_decode_is_the_last_row_of_the_forward_pass(alpha, oracle):
    """q of one token at the end of a causal sequence sees every key: the forward oracle's last
    row, from scattered pages."""
    import torch
    rng = np.random.default_rng(3)
    Hq, Hkv, d, P = 4, 2, 64, 5
    lens = [23, 0, 1, 10]
    kc = rng.standard_normal((12, Hkv, P, d)).astype(np.float32)
    vc = rng.standard_normal((12, Hkv, P, d)).astype(np.float32)
    ids = rng.permutation(12)
    tables = np.zeros((4, 5), dtype=int)
    tables[0], tables[2, 0], tables[3, :2] = ids[:5], ids[5], ids[6:8]
    q = rng.standard_normal((4, Hq, d)).astype(np.float32)
    a32 = orc.alpha_as_float32(alpha)
    o, tau = paged.decode(q.astype(float), kc.astype(float), vc.astype(float), tables, lens, a32)
    for b, n in enumerate(lens):
        if n == 0:
            assert (o[b] == 0).all() and np.isinf(tau[b]).all()
            continue
        full = np.zeros((1, Hq, n, d), dtype=np.float32)
        full[0, :, -1] = q[b]
        k, v = paged.gather(kc, tables[b], n), paged.gather(vc, tables[b], n)
        ref = oracle.attention_rows(torch.from_numpy(full), torch.from_numpy(k.copy())[None],
                                    torch.from_numpy(v.copy())[None], a32, True)
        ro = np.asarray(ref["out"]).reshape(Hq, n, d)[:, -1]
        rt = np.asarray(ref["tau"]).reshape(Hq, n)[:, -1]
        # the oracle takes alpha as a double; both are fp64 sums of n <= 23 terms
        np.testing.assert_allclose(o[b], ro, rtol=0, atol=1e-6)
        np.testing.assert_allclose(tau[b], rt, rtol=0, atol=1e-6)
