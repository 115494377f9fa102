"""Cases of the serving operators around a paged key-value cache, with their plain forms.

    page tables   grow the requests' block tables from a free list and give every new token its slot
    cache append  store the new tokens' keys and values in the slots
    decode        alpha-entmax attention of one new token per request over its paged keys

A case is a dict of plain values; `prepare` makes its inputs on the GPU, `run` is one pass (the
plain torch form, or with `own` the framework's call), `exact` the definition in 64 bits and `work`
what a pass cannot do without.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases --

def listed():
    return [
        # One decoding step of a full batch: every request grows by one token, most without a
        # new page.  Latency is all there is to it.
        dict(name="tables_step_b64", op="tables", B=64, lens="log", min_len=1, max_len=16384,
             new="one", page=16, padded=True, lens_seed=11),
        # The packed 32K batch arrives for prefill: four prompts, empty tables.
        dict(name="tables_prefill_32k", op="tables", B=4, lens="0,0,0,0",
             new="1000,3000,8192,20000", page=64, padded=False, lens_seed=0),
        # A server with a thousand requests mid-way through chunked prefill and decoding.
        dict(name="tables_mixed_b1000", op="tables", B=1000, lens="log", min_len=1,
             max_len=8191, new="log", max_new=2048, page=16, padded=False, lens_seed=12),
        # The new tokens of one decoding step.
        dict(name="append_step_b64", op="append", B=64, T=1, Hkv=8, d=128, page=64, dtype="bf16",
             layout="heads", padded=True, drop=0.05),
        # The keys and values of the packed 32K prefill, cache with tokens before heads.
        dict(name="append_prefill_32k", op="append", B=1, T=32192, Hkv=8, d=128, page=16,
             dtype="bf16", layout="tokens", padded=False, drop=0.0),
        # A batch of 4K prompts in fp32 with small heads and pages of an odd size.
        dict(name="append_4k_fp32", op="append", B=3, T=4095, Hkv=8, d=64, page=24, dtype="fp32",
             layout="heads", padded=True, drop=0.02),
        # A single user's request early in its life: latency counts.
        dict(name="decode_b1_1k", op="decode", B=1, Hq=32, Hkv=8, d=128, dtype="bf16", page=16,
             lens="1000", alpha=1.5, spike_frac=0.02, spike_scale=4.0, layout="heads",
             fused_q=False, lens_seed=0),
        # A single request with a 128K context: the cache has to be split over the whole GPU.
        dict(name="decode_b1_128k", op="decode", B=1, Hq=32, Hkv=8, d=128, dtype="bf16", page=64,
             lens="131072", alpha=1.5, spike_frac=0.01, spike_scale=5.0, layout="heads",
             fused_q=False, lens_seed=0),
        # A full batch of ragged contexts up to 16K, sparsemax: the throughput case.
        dict(name="decode_b64_16k", op="decode", B=64, Hq=32, Hkv=8, d=128, dtype="bf16", page=64,
             lens="uniform", min_len=8000, max_len=16384, alpha=2.0, spike_frac=0.02,
             spike_scale=4.0, layout="tokens", fused_q=True, lens_seed=13),
        # The packed 32K batch's lengths without key spikes at alpha = 1.333: wide supports.
        dict(name="decode_ragged_32k", op="decode", B=4, Hq=32, Hkv=8, d=128, dtype="bf16",
             page=16, lens="1000,3000,8192,20000", alpha=1.333, spike_frac=0.0, spike_scale=1.0,
             layout="heads", fused_q=False, lens_seed=0),
        # Small heads without grouping, some rows of the batch unused (length 0).
        dict(name="decode_b33_4k_d64", op="decode", B=33, Hq=8, Hkv=8, d=64, dtype="bf16",
             page=32, lens="ragged0", min_len=1, max_len=4096, alpha=1.5, spike_frac=0.02,
             spike_scale=4.0, layout="heads", fused_q=True, lens_seed=14),
        # True fp32.
        dict(name="decode_b4_4k_fp32", op="decode", B=4, Hq=8, Hkv=2, d=64, dtype="fp32", page=16,
             lens="uniform", min_len=200, max_len=4096, alpha=1.5, spike_frac=0.0,
             spike_scale=1.0, layout="heads", fused_q=False, lens_seed=15),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: the same operators, types, layouts and options over the whole range."""
    op = rng.choice(["tables", "append", "decode", "decode"])
    seed = rng.randrange(1 << 30)
    if op == "tables":
        c = dict(op=op, B=_log_int(rng, 1, 1000), lens="log", min_len=1,
                 max_len=_log_int(rng, 2, 16384), new=rng.choice(["one", "log"]),
                 max_new=_log_int(rng, 1, 2048), page=rng.choice([1, 8, 16, 24, 32, 64, 128]),
                 padded=rng.random() < 0.4, lens_seed=seed)
        return c
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    d = rng.choice([64, 128])
    layout = rng.choice(["heads", "tokens"])
    page = rng.choice([1, 8, 16, 24, 32, 64, 128])
    if op == "append":
        Hkv = rng.choice([1, 2, 3, 8])
        N = _log_int(rng, 1, 32192)
        padded = rng.random() < 0.5
        B = _log_int(rng, 1, min(64, N)) if padded else 1
        return dict(op=op, B=B, T=max(1, N // B), Hkv=Hkv, d=d, page=page, dtype=dtype,
                    layout=layout, padded=padded, drop=rng.choice([0.0, 0.1]))
    Hkv = rng.choice([1, 2, 3, 8])
    G = rng.choice([1, 2, 4, 5, 8, 16])
    max_len = _log_int(rng, 1, 131072)
    # keys over all heads within a quarter of the largest listed case
    room = (64 * 12000 * 8 * 256) // 4 // (Hkv * d * (4 if dtype == "fp32" else 2))
    B = _log_int(rng, 1, max(1, min(64, room // max_len)))
    spikes = rng.choice([(0.0, 1.0), (0.02, 4.0), (0.01, 5.0)])
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, dtype=dtype, page=page,
                lens=rng.choice(["uniform", "ragged0", "log"]), min_len=1, max_len=max_len,
                alpha=rng.choice([1.333, 1.5, 2.0]), spike_frac=spikes[0], spike_scale=spikes[1],
                layout=layout, fused_q=rng.random() < 0.5, lens_seed=seed)


def _lens(case, spec=None):
    spec = case["lens"] if spec is None else spec
    rng = random.Random(case["lens_seed"])
    B = case["B"]
    if spec == "uniform":
        return [rng.randint(case["min_len"], case["max_len"]) for _ in range(B)]
    if spec == "log":
        return [_log_int(rng, case["min_len"], case["max_len"]) for _ in range(B)]
    if spec == "ragged0":  # about one row in eight is unused
        return [0 if rng.random() < 0.125 else rng.randint(case["min_len"], case["max_len"])
                for _ in range(B)]
    return [int(x) for x in spec.split(",")]


def _new_lens(case):
    if case["new"] == "one":
        return [1] * case["B"]
    if case["new"] == "log":  # requests that decode beside requests that prefill a chunk
        rng = random.Random(case["lens_seed"] + 1)
        return [0 if rng.random() < 0.1 else _log_int(rng, 1, case["max_new"])
                for _ in range(case["B"])]
    return [int(x) for x in case["new"].split(",")]


def _blocks(n, page):
    return -(-n // page)


def work(case):
    """Bytes and operations of one pass that no implementation can do without."""
    if case["op"] == "tables":
        lens, new = _lens(case), _new_lens(case)
        B, P = case["B"], case["page"]
        rows = max(1, B * max(new) if case["padded"] else sum(new))
        taken = sum(_blocks(a + n, P) - _blocks(a, P) for a, n in zip(lens, new))
        # lengths in and out, offsets out, free pages in, table entries out, slots out
        return {"bytes": 4 * (2 * B + B + B + 2) + 8 * taken + 8 * rows, "flops": 2 * B + rows}
    esz = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "append":
        n = case["B"] * case["T"]
        return {"bytes": 8 * n + 4 * n * case["Hkv"] * case["d"] * esz, "flops": 0}
    lens = _lens(case)
    rows = case["B"] * case["Hq"]
    # every key once, the page numbers, q in, out and tau out, and of the values one row at least
    # per query (which others are read depends on the data: only keys with p > 0)
    live = sum(1 for n in lens if n)
    by = sum(lens) * case["Hkv"] * case["d"] * esz + 4 * sum(_blocks(n, case["page"]) for n in lens)
    by += 2 * rows * case["d"] * esz + 4 * rows + live * case["Hq"] * case["d"] * esz
    return {"bytes": by, "flops": 2 * sum(lens) * case["Hq"] * case["d"]}


# ------------------------------------------------------------------------------------ inputs --

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(g, pages, Hkv, P, d, dtype, layout):
    """A cache [pages, Hkv, P, d] of N(0, 1) values; "tokens" stores a page's tokens before its
    heads and is seen through a transposed view."""
    shape = (pages, Hkv, P, d) if layout == "heads" else (pages, P, Hkv, d)
    c = torch.randn(shape, generator=g, dtype=dtype, device="cuda")
    return c if layout == "heads" else c.transpose(1, 2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "tables":
        lens, new = _lens(case), _new_lens(case)
        B, P = case["B"], case["page"]
        have = [_blocks(n, P) for n in lens]
        need = [_blocks(a + n, P) for a, n in zip(lens, new)]
        W = max(need) + 1
        total = sum(need) + 8
        ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        live = torch.arange(W, device="cuda")[None, :] < _i32(have)[:, None]
        used = sum(have)
        table[live] = ids[:used]
        start = int(torch.randint(0, 4, (1,), generator=g, device="cuda"))
        free = torch.cat([ids[used:used + start], ids[used:]])  # `start` entries already taken
        rows = max(1, max(new) if case["padded"] else sum(new))
        return dict(case=case, lens=_i32(lens), new=_i32(new), free=free, start=_i32([start]),
                    table=table, rows=rows)
    dtype = DTYPES[case["dtype"]]
    Hkv, d, P = case["Hkv"], case["d"], case["page"]
    if case["op"] == "append":
        B, T = case["B"], case["T"]
        n = B * T
        pages = _blocks(n, P) + 3
        kc = _cache(g, pages, Hkv, P, d, dtype, case["layout"])
        vc = _cache(g, pages, Hkv, P, d, dtype, case["layout"])
        order = torch.randperm(pages, generator=g, device="cuda")
        pos = torch.arange(n, device="cuda")
        slots = order[pos // P] * P + pos % P
        if case["drop"]:  # padding rows
            slots[torch.rand(n, generator=g, device="cuda") < case["drop"]] = -1
        shape = (B, Hkv, T, d) if case["padded"] else (Hkv, n, d)
        k = torch.randn(shape, generator=g, dtype=dtype, device="cuda")
        v = torch.randn(shape, generator=g, dtype=dtype, device="cuda")
        return dict(case=case, k=k, v=v, kc=kc, vc=vc, slots=slots)
    lens = _lens(case)
    B, Hq = case["B"], case["Hq"]
    nb = [_blocks(n, P) for n in lens]
    W = max(1, max(nb))
    pages = sum(nb) + 2
    kc = _cache(g, pages, Hkv, P, d, dtype, case["layout"])
    vc = _cache(g, pages, Hkv, P, d, dtype, case["layout"])
    if case["spike_frac"]:
        hit = torch.rand((pages, Hkv, P, 1), generator=g, device="cuda") < case["spike_frac"]
        kc.mul_(1 + (case["spike_scale"] - 1) * hit.to(dtype))
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(W, device="cuda")[None, :] < _i32(nb)[:, None]] = ids[:sum(nb)]
    if case["fused_q"]:  # q as the leading columns of a fused projection's output
        q = torch.randn((B, (Hq + 2 * Hkv) * d), generator=g, dtype=dtype, device="cuda")
        q = q[:, :Hq * d].view(B, Hq, d)
    else:
        q = torch.randn((B, Hq, d), generator=g, dtype=dtype, device="cuda")
    return dict(case=case, q=q, kc=kc, vc=vc, table=table, lens=_i32(lens), host_lens=lens,
                max_len=max(lens), workspace=_workspace(case, q, kc, max(1, max(lens))))


def _workspace(case, q, kc, max_len):
    """The scratch memory a serving program keeps beside its cache."""
    if not own:
        return None
    import adaptive_sparse_attention_b200 as ea
    return ea.alloc_decode_workspace(q, kc, max_len)


# --------------------------------------------------------------------------------- one pass --

def run(state):
    op = state["case"]["op"]
    if own:
        import adaptive_sparse_attention_b200 as ea
        c = state["case"]
        if op == "tables":
            slots, lens, cu, nxt = ea.page_tables(state["lens"], state["new"], state["free"],
                                                  state["start"], state["table"], c["page"],
                                                  state["rows"], padded=c["padded"])
            return [state["table"], slots, lens, cu, nxt]
        if op == "append":
            ea.paged_append(state["k"], state["v"], state["kc"], state["vc"], state["slots"])
            return [state["kc"], state["vc"]]
        out, tau = ea.entmax_attn_decode(state["q"], state["kc"], state["vc"], state["table"],
                                         state["lens"], c["alpha"], max_len=state["max_len"],
                                         workspace=state["workspace"])
        return [out, tau]
    return {"tables": _plain_tables, "append": _plain_append, "decode": _plain_decode}[op](state)


def _plain_tables(s):
    """table[b, have_b + i] = free[start + first_b + i] and, per new token at position pos,
    slot = table[b, pos // P] * P + pos % P (-1 past the last new token)."""
    c, P, table = s["case"], s["case"]["page"], s["table"]
    lens, new = s["lens"], s["new"]
    W = table.shape[1]
    have, total = (lens + P - 1) // P, lens + new
    need = (total + P - 1) // P
    take = need - have
    ends = torch.cumsum(take, 0)
    col = torch.arange(W, device="cuda")[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    at = s["start"].long() + (ends - take)[:, None] + col - have[:, None]
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    cu = torch.zeros(c["B"] + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(new, 0)
    if c["padded"]:
        t = torch.arange(s["rows"], device="cuda")[None, :].expand(c["B"], -1)
        row = torch.arange(c["B"], device="cuda")[:, None].expand_as(t)
        live = t < new[:, None]
    else:
        n = torch.arange(s["rows"], device="cuda")
        row = (torch.searchsorted(cu, n.to(torch.int32), right=True) - 1).clamp(0, c["B"] - 1)
        t = n - cu[row]
        live = t < new[row]
    pos = lens[row].long() + t
    page = table[row, (pos // P).clamp(max=W - 1)].long()
    slots = torch.where(live, page * P + pos % P, torch.full_like(pos, -1))
    return [table, slots, total, cu, (s["start"] + ends[-1]).to(torch.int32)]


def _plain_append(s):
    """cache[slot // P, h, slot % P] = new[token, h] for the tokens with a slot."""
    P = s["case"]["page"]
    Hkv, d = s["kc"].shape[1], s["kc"].shape[3]
    live = s["slots"] >= 0
    slot = s["slots"][live]
    for new, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
        rows = new if new.dim() == 3 else new.transpose(0, 1).reshape(Hkv, -1, d)
        cache[slot // P, :, slot % P] = rows[:, live].transpose(0, 1)
    return [s["kc"], s["vc"]]


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))  # the library takes alpha as a float


def _pages_of(cache, table, b, n):
    """The first n keys (values) of request b: [Hkv, n, d]."""
    P = cache.shape[2]
    rows = cache[table[b, :_blocks(n, P)].long()]
    return rows.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]


def _power(x, beta):
    if beta == 1.0:
        return x
    return x * x if beta == 2.0 else x ** beta


def _plain_decode(s):
    """z = (alpha - 1) q . k / sqrt(d), p = [z - tau]_+^(1 / (alpha - 1)) with sum p = 1, o = p v;
    tau by bisection, in 64 bits because z - tau cancels."""
    c, lens = s["case"], s["host_lens"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    am1 = _f32(c["alpha"]) - 1.0
    beta = 1.0 / am1
    z = torch.full((B, Hq, max(1, max(lens))), -math.inf, device="cuda")
    for b, n in enumerate(lens):
        if n:
            k = _pages_of(s["kc"], s["table"], b, n).float()
            q = s["q"][b].float().view(Hkv, Hq // Hkv, d)
            z[b, :, :n] = (q @ k.transpose(1, 2)).view(Hq, n) * (am1 / math.sqrt(d))
    top = z.amax(-1, keepdim=True).double()
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))  # unused rows
    lo, hi = top - 1.0, top.clone()
    for _ in range(52):
        mid = 0.5 * (lo + hi)
        big = _power((z - mid).clamp_min_(0.0), beta).sum(-1, keepdim=True) > 1.0
        lo, hi = torch.where(big, mid, lo), torch.where(big, hi, mid)
    tau = 0.5 * (lo + hi)
    p = _power((z - tau).clamp_min_(0.0), beta).float()
    out = torch.zeros((B, Hq, d), device="cuda")
    for b, n in enumerate(lens):
        if n:
            v = _pages_of(s["vc"], s["table"], b, n).float()
            out[b] = (p[b, :, :n].view(Hkv, -1, n) @ v).view(Hq, d)
    tau = tau[..., 0].float()
    tau[s["lens"] == 0] = math.inf
    return [out.to(s["q"].dtype), tau]


# ------------------------------------------------------------------------- 64-bit definition --

def exact(case, seed):
    """For a decoding case the outputs in 64 bits, tau from the sorted scores; the page tables are
    whole numbers and the append moves bits, so those have no computed value."""
    if case["op"] != "decode":
        return None
    s = prepare(case, seed)
    alpha = _f32(case["alpha"])
    Hkv, G, d, P = case["Hkv"], case["Hq"] // case["Hkv"], case["d"], case["page"]
    outs, taus = [], []
    for b, n in enumerate(_lens(case)):
        if n == 0:
            outs.append(torch.zeros((case["Hq"], d), dtype=torch.float64, device="cuda"))
            taus.append(torch.full((case["Hq"],), math.inf, dtype=torch.float64, device="cuda"))
            continue
        pos = torch.arange(n, device="cuda")
        page, off = s["table"][b].long()[pos // P], pos % P
        for h in range(Hkv):
            k = s["kc"][page, h, off].double()
            v = s["vc"][page, h, off].double()
            z = (s["q"][b, h * G:(h + 1) * G].double() @ k.T) / math.sqrt(d) * (alpha - 1.0)
            tau = _sorted_tau(z, alpha)
            p = torch.relu(z - tau[:, None]).pow(1.0 / (alpha - 1.0))
            outs.append(p @ v)
            taus.append(tau)
    return [torch.cat(outs).view(case["B"], case["Hq"], d), torch.cat(taus).view(case["B"], -1)]


def _sorted_tau(z, alpha):
    """tau of each row: with the scores in falling order the support is the longest prefix whose
    mass at its own last score stays below 1; on it the sum is solved for tau."""
    beta = 1.0 / (alpha - 1.0)
    zs = torch.sort(z, dim=-1, descending=True).values
    n = zs.shape[-1]
    r = torch.arange(1, n + 1, dtype=torch.float64, device=z.device)
    shift = zs - zs[:, :1]  # the largest score as the origin: no cancellation in the sums
    s1, s2 = torch.cumsum(shift, -1), torch.cumsum(shift * shift, -1)
    if alpha == 2.0:
        k = (s1 - r * shift < 1.0).sum(-1, keepdim=True)
        t = (s1.gather(-1, k - 1) - 1.0) / k
    elif alpha == 1.5:
        k = (s2 - 2.0 * shift * s1 + r * shift * shift < 1.0).sum(-1, keepdim=True)
        mean, sq = s1.gather(-1, k - 1) / k, s2.gather(-1, k - 1) / k
        t = mean - torch.sqrt((1.0 / k - (sq - mean * mean)).clamp_min(0.0))
    else:  # Newton's steps from the left on sum (z - tau)^beta = 1, convex in tau
        t = torch.full_like(zs[:, :1], -1.0)
        for _ in range(80):
            x = torch.relu(shift - t)
            f = x.pow(beta).sum(-1, keepdim=True) - 1.0
            t = t + f / (beta * x.pow(beta - 1.0).sum(-1, keepdim=True))
    return (t + zs[:, :1])[:, 0]
