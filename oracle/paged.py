"""Oracle of the paged key-value cache, in plain Python and numpy fp64, sharing no code with the
CUDA path: the page tables request by request, the append row by row, and alpha-entmax attention of
one token per request with the oracle's exact tau."""
from __future__ import annotations

import numpy as np

from . import oracle as orc


def page_tables(lens, new_lens, free_pages, free_start, tables, page, n_new, padded=False):
    """(tables, slots, lens_out, cu_new, free_next), all new arrays.  Requests are served in
    order; the takes of every request whose lengths fit its table row are laid out one after the
    other in the free list, whether or not the list is long enough for them."""
    tables = np.array(tables, dtype=np.int64)
    B, W = tables.shape
    n_free = len(free_pages)
    room = n_free - free_start if 0 <= free_start <= n_free else 0
    slots = np.full((B, n_new) if padded else (n_new,), -1, dtype=np.int64)
    lens_out = np.array(lens, dtype=np.int64)
    cu = np.zeros(B + 1, dtype=np.int64)
    at = taken = 0
    for b in range(B):
        old, add = int(lens[b]), int(new_lens[b])
        cu[b + 1] = cu[b] + max(add, 0)
        if old < 0 or add < 0 or old + add > W * page or (padded and add > n_new):
            continue
        have, need = -(-old // page), -(-(old + add) // page)
        first, at = at, at + need - have
        if not padded and cu[b + 1] > n_new:
            continue
        if need > have and at > room:
            continue
        for i in range(need - have):
            tables[b, have + i] = free_pages[free_start + first + i]
        if need > have:
            taken = at
        lens_out[b] = old + add
        for t in range(add):
            pg = tables[b, (old + t) // page]
            where = (b, t) if padded else cu[b] + t
            if pg >= 0:
                slots[where] = pg * page + (old + t) % page
    return tables, slots, lens_out, cu, free_start + taken


def append(cache, rows, slots):
    """cache [pages, Hkv, P, d] with rows [Hkv, N, d] stored in slots [N] (a copy)."""
    out = np.array(cache)
    P = out.shape[2]
    for n, s in enumerate(slots):
        if 0 <= s < out.shape[0] * P:
            out[s // P, :, s % P] = rows[:, n]
    return out


def decode_rows(q, k, v, alpha):
    """One kv head: q [G, d], k and v [n, d] in fp64.  Returns o, tau and z, the scores."""
    z = (alpha - 1.0) * (q @ k.T) / np.sqrt(q.shape[1])
    o = np.zeros_like(q)
    tau = np.zeros(q.shape[0])
    for g in range(q.shape[0]):
        p, tau[g] = orc.entmax_vec(z[g], alpha)
        o[g] = p @ v
    return o, tau, z


def gather(cache, table, n):
    """The first n rows of a request: [Hkv, n, d]."""
    P = cache.shape[2]
    j = np.arange(n)
    return cache[np.asarray(table)[j // P], :, j % P].transpose(1, 0, 2)


def decode(q, k_cache, v_cache, tables, lens, alpha):
    """q [B, Hq, d], caches [pages, Hkv, P, d], all fp64.  Returns (o [B, Hq, d], tau [B, Hq])."""
    B, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    o, tau = np.zeros((B, Hq, d)), np.full((B, Hq), np.inf)
    for b in range(B):
        if lens[b] == 0:
            continue
        k, v = gather(k_cache, tables[b], lens[b]), gather(v_cache, tables[b], lens[b])
        for h in range(Hkv):
            s = slice(h * G, (h + 1) * G)
            o[b, s], tau[b, s], _ = decode_rows(q[b, s], k[h], v[h], alpha)
    return o, tau


def decode_bounds(q, k_cache, v_cache, tables, lens, alpha, tau, eps_out, n_steps_ulps=8):
    """Error bounds (of o per element, of tau per row) of an fp32 computation with outputs of
    relative rounding eps_out / 2, from the rounding of its parts (u = 2^-24):
      a score sums d products: |dz| <= (2 d + 4) u c sum |q_e k_e| (each addition truncated, 2 u);
      tau is 1-Lipschitz in the scores (max norm), found to n_steps_ulps units of 2 u max(|tau|, 1);
      p = x^beta with |dx| <= 2 dz + dtau: |dp| <= beta (x + dx)^(beta - 1) dx for beta >= 1, and
      dx^beta for beta < 1, plus 64 u p for the power;
      o sums n products p v: (n + 2) u sum p |v| more, then its rounding.
    """
    u = 2.0 ** -24
    B, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    beta = 1.0 / (alpha - 1.0)
    c = (alpha - 1.0) / np.sqrt(d)
    bo, bt = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        if lens[b] == 0:
            continue
        k, v = gather(k_cache, tables[b], lens[b]), gather(v_cache, tables[b], lens[b])
        for hq in range(Hq):
            h = hq // G
            z = c * (k[h] @ q[b, hq])
            dz = (2 * d + 4) * u * c * (np.abs(k[h]) @ np.abs(q[b, hq]))
            near = z > z.max() - 1.1
            dz = dz[near].max()
            dt = dz + n_steps_ulps * 2 * u * max(abs(tau[b, hq]), 1.0)
            dx = dz + dt
            x = z - tau[b, hq]
            live = x > -dx
            xl = np.maximum(x[live], 0.0)
            p = xl ** beta
            if beta >= 1.0:
                dp = beta * (xl + dx) ** (beta - 1.0) * dx
            else:
                dp = np.full_like(p, dx ** beta)
            dp = dp + 64 * u * p
            va = np.abs(v[h][live])
            err = dp @ va + (live.sum() + 2) * u * (p @ va)
            o = np.abs(p @ v[h][live])
            bo[b, hq] = err + (o + err) * eps_out / 2
            bt[b, hq] = dt + u * abs(tau[b, hq])
    return bo, bt
