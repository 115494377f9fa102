"""entmax_attn_status with several conditions latched: a pass that gave up and an index out of
range, in either order, are both reported, the pass first."""
import pytest
import torch

import adaptive_sparse_attention_b200 as ea
from adaptive_sparse_attention_b200 import _native
from adaptive_sparse_attention_b200.workloads import random_case

pytestmark = pytest.mark.gpu


def give_up():
    """A tau pass whose query tile is never requested: its bounded waits run out."""
    _, inputs = random_case(B=1, Hq=1, Hkv=1, T=128, d=64, dtype="bf16", alpha=1.5, name="stall",
                            seed=5)
    q, k, v, cu = (x.cuda() if x is not None else None for x in inputs)
    _, tau, mask = ea.alloc_outputs(q, k, None)
    ea.tau_pass(q, k, tau, mask, ea.alloc_workspace(q, k, None), 1.5, 10, True, None,
                _native.FLAG_TEST_STALL)


def out_of_range():
    kc = torch.zeros(2, 1, 16, 64, device="cuda")
    k = torch.zeros(1, 1, 64, device="cuda")
    ea.paged_append(k, k, kc, kc.clone(), torch.tensor([32], device="cuda"))


@pytest.mark.parametrize("order", ["range last", "timeout last"])
def test_neither_condition_hides_the_other(order):
    assert ea.status() == _native.OK
    first, second = (give_up, out_of_range) if order == "range last" else (out_of_range, give_up)
    first()
    second()
    assert ea.status() == _native.ETIMEOUT
    assert ea.status() == _native.ERANGE
    assert ea.status() == _native.OK


def test_each_condition_alone():
    for act, code in ((out_of_range, _native.ERANGE), (give_up, _native.ETIMEOUT)):
        act()
        act()
        assert ea.status() == code and ea.status() == _native.OK
