"""Host-only checks of the paged-cache entry points: argument errors are reported before any
launch, and the workspace query answers as documented."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def native():
    from adaptive_sparse_attention_b200 import build, _native
    build.build()
    return _native


def _p(x):
    return ctypes.c_void_p(x) if x else None


TABLES = dict(lens=0x1000, new=0x2000, free=0x3000, n_free=8, start=0x4000, tables=0x5000, stride=4,
              W=4, B=2, page=16, slots=0x6000, n_new=3, padded=0, lens_out=0x7000, cu=0x8000,
              next=0x9000)


@pytest.mark.parametrize("change,code", [
    (dict(lens=0), 1), (dict(new=0), 1), (dict(free=0), 1), (dict(start=0), 1),
    (dict(tables=0), 1), (dict(slots=0), 1), (dict(lens_out=0), 1), (dict(cu=0), 1),
    (dict(next=0), 1), (dict(n_free=-1), 1), (dict(W=0), 1), (dict(B=0), 1), (dict(B=8193), 1),
    (dict(stride=3), 1), (dict(page=0), 1), (dict(n_new=0), 1), (dict(padded=2), 1),
    (dict(lens_out=0x1000), 1), (dict(lens_out=0x2000), 1), (dict(next=0x4000), 1),
    (dict(B=8192, W=1 << 18, stride=1 << 18), 1), (dict(slots=0x6004), 2), (dict(lens=0x1002), 2),
    (dict(tables=0x5001), 2)])
def test_page_tables_refusals(native, change, code):
    a = dict(TABLES, **change)
    rc = native.lib().entmax_attn_page_tables(
        _p(a["lens"]), _p(a["new"]), _p(a["free"]), a["n_free"], _p(a["start"]), _p(a["tables"]),
        a["stride"], a["W"], a["B"], a["page"], _p(a["slots"]), a["n_new"], a["padded"],
        _p(a["lens_out"]), _p(a["cu"]), _p(a["next"]), None)
    assert rc == code


APPEND = dict(k=0x1000, v=0x2000, sb=0, sh=640, st=128, kc=0x3000, vc=0x4000, ps=4096, hs=2048,
              ss=128, pages=4, page=16, slots=0x5000, B=1, Hkv=2, T=5, d=128, dtype=1)


@pytest.mark.parametrize("change,code", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(kc=0), 1), (dict(vc=0), 1), (dict(slots=0), 1),
    (dict(B=0), 1), (dict(T=0), 1), (dict(Hkv=0), 1), (dict(B=1 << 16, T=1 << 15), 1),
    (dict(d=96), 1), (dict(dtype=2), 1), (dict(pages=0), 1), (dict(page=0), 1),
    (dict(ss=64), 1), (dict(hs=0), 1), (dict(ps=100), 1), (dict(ps=4100), 1), (dict(st=132), 1),
    (dict(sh=-640), 1), (dict(k=0x1008), 2), (dict(vc=0x4002), 2), (dict(slots=0x5004), 2)])
def test_append_refusals(native, change, code):
    a = dict(APPEND, **change)
    rc = native.lib().entmax_attn_paged_append(
        _p(a["k"]), _p(a["v"]), a["sb"], a["sh"], a["st"], _p(a["kc"]), _p(a["vc"]), a["ps"],
        a["hs"], a["ss"], a["pages"], a["page"], _p(a["slots"]), a["B"], a["Hkv"], a["T"], a["d"],
        a["dtype"], None)
    assert rc == code


DECODE = dict(q=0x1000, qb=512, qh=128, kc=0x3000, vc=0x4000, ps=4096, hs=2048, ss=128, pages=4,
              page=16, tables=0x5000, stride=4, W=4, lens=0x6000, out=0x7000, tau=0x8000,
              ws=0x10000, ws_bytes=1 << 40, B=2, Hq=4, Hkv=2, max_len=64, d=128, alpha=1.5,
              n_iter=10, dtype=1)


@pytest.mark.parametrize("change,code", [
    (dict(q=0), 1), (dict(kc=0), 1), (dict(vc=0), 1), (dict(tables=0), 1), (dict(lens=0), 1),
    (dict(out=0), 1), (dict(tau=0), 1), (dict(ws=0), 1), (dict(B=0), 1), (dict(B=8193), 1),
    (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(W=0), 1), (dict(stride=3), 1), (dict(max_len=0), 1),
    (dict(max_len=65), 1), (dict(d=32), 1), (dict(alpha=1.0), 1), (dict(alpha=float("nan")), 1),
    (dict(alpha=float("inf")), 1), (dict(n_iter=0), 1), (dict(n_iter=1001), 1),
    (dict(dtype=-1), 1), (dict(qh=132), 1), (dict(qb=-8), 1), (dict(ss=120), 1),
    (dict(hs=2052), 1), (dict(q=0x1008), 2), (dict(kc=0x3008), 2), (dict(out=0x7004), 2),
    (dict(tables=0x5002), 2), (dict(lens=0x6001), 2), (dict(tau=0x8002), 2),
    (dict(ws=0x10080), 2), (dict(ws_bytes=1000), 5)])
def test_decode_refusals(native, change, code):
    a = dict(DECODE, **change)
    rc = native.lib().entmax_attn_decode(
        _p(a["q"]), a["qb"], a["qh"], _p(a["kc"]), _p(a["vc"]), a["ps"], a["hs"], a["ss"],
        a["pages"], a["page"], _p(a["tables"]), a["stride"], a["W"], _p(a["lens"]), _p(a["out"]),
        _p(a["tau"]), _p(a["ws"]), a["ws_bytes"], a["B"], a["Hq"], a["Hkv"], a["max_len"],
        a["d"], a["alpha"], a["n_iter"], a["dtype"], None)
    assert rc == code


def test_workspace_query(native):
    f = native.lib().entmax_attn_decode_workspace_bytes
    assert f(0, 4, 2, 16) == f(1, 3, 2, 16) == f(1, 4, 0, 16) == f(1, 4, 2, 0) == 0
    assert f(8193, 4, 2, 16) == 0 and f(8192, 4, 4, (1 << 31) - 1) == 0
    assert 0 < f(1, 1, 1, 1) <= f(1, 4, 1, 1) <= f(1, 4, 1, 1000) < f(8, 4, 1, 1000)
    assert f(1, 4, 2, 131072) > 1 and f(64, 32, 8, 131072) > 1 << 31  # 64-bit sizes


def test_strerror_of_the_new_code(native):
    assert b"range" in native.lib().entmax_attn_strerror(native.ERANGE)


def test_binding_refuses_host_tensors():
    import torch

    import adaptive_sparse_attention_b200 as ea
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(4, 2, 16, 64)
    with pytest.raises(ValueError):
        ea.page_tables(i, i, i, i[:1], i.view(2, 1), 16, 4)
    with pytest.raises(ValueError):
        ea.paged_append(torch.zeros(2, 3, 64), torch.zeros(2, 3, 64), c, c,
                        torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        ea.entmax_attn_decode(torch.zeros(2, 4, 64), c, c, i.view(2, 1), i)
