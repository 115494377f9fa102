"""The C entry points from several host threads at once (ctypes releases the interpreter's lock),
on streams of their own."""
import threading

import pytest
import torch

from adaptive_sparse_attention_b200 import _native

pytestmark = pytest.mark.gpu


def test_page_tables_of_different_batches_at_once():
    """Batches of thousands of requests take more shared memory than a kernel has by default: what one
    thread's call allows must not be taken from another's."""
    lib = _native.lib()
    codes, states = {}, {}

    def state(B):
        z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
        s = dict(lens=z(B), new=torch.ones(B, dtype=torch.int32, device="cuda"),
                 free=torch.arange(B, dtype=torch.int32, device="cuda"), start=z(1), tables=z(B),
                 slots=z(B, torch.int64), out=z(B), cu=z(B + 1), next=z(1),
                 stream=torch.cuda.Stream())
        states[B] = s
        return s

    def calls(B, n):
        p = {k: (x.cuda_stream if k == "stream" else x.data_ptr()) for k, x in states[B].items()}
        codes[B] = [lib.entmax_attn_page_tables(
            p["lens"], p["new"], p["free"], B, p["start"], p["tables"], 1, 1, B, 16, p["slots"], B,
            0, p["out"], p["cu"], p["next"], p["stream"]) for _ in range(n)]

    sizes = (8192, 3200, 5000)
    for B in sizes:
        state(B)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=calls, args=(B, 3000)) for B in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for B in sizes:
        assert set(codes[B]) == {_native.OK}, (B, {c: codes[B].count(c) for c in set(codes[B])})
        s = states[B]
        assert s["out"].eq(1).all() and int(s["next"]) == B
        assert torch.equal(s["slots"], 16 * torch.arange(B, device="cuda"))
