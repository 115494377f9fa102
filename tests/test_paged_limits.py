"""Host checks of the paged-cache entry points at the largest sizes (no GPU, nothing is launched)."""
import pytest


@pytest.fixture(scope="module")
def native():
    from adaptive_sparse_attention_b200 import build, _native
    build.build()
    return _native


def device_int32(x):
    """x as the kernels' 32-bit arithmetic has it."""
    return (x + (1 << 31)) % (1 << 32) - (1 << 31)


def test_longest_request(native):
    """Lengths are cut into units of 16 keys and the join steps through 32 keys at a time, 32 lists
    at once, eight steps ahead, all in 32 bits: what they reach past the longest length allowed
    must stay below 2^31.  2^31 - 1 did not: rounding it up to units gave a negative count."""
    f = native.lib().entmax_attn_decode_workspace_bytes
    assert device_int32(((1 << 31) - 1) + 15) >> 4 < 0
    limit = (1 << 31) - 4096
    assert f(1, 1, 1, limit) > 8 * limit
    for n in (limit + 1, (1 << 31) - 16, (1 << 31) - 15, (1 << 31) - 1):
        assert f(1, 1, 1, n) == 0
    units = (limit + 15) >> 4
    assert device_int32(units * 16) == units * 16
    reach = limit + 32 * 32 + 8 * 32 + 32  # every list rounded up to 32, eight steps, the lanes
    assert device_int32(reach) == reach


def test_largest_slot_map(native):
    import ctypes
    p = ctypes.c_void_p
    for n_new in ((1 << 31) - 4, (1 << 31) - 1):
        assert native.lib().entmax_attn_page_tables(
            p(0x1000), p(0x2000), p(0x3000), 8, p(0x4000), p(0x5000), 4, 4, 2, 16, p(0x6000),
            n_new, 0, p(0x7000), p(0x8000), p(0x9000), None) == native.EINVAL


def test_wrapped_token_sums_would_leave_the_tables():
    """Why the device's sums of new_lens must stop at 2^31 - 1: with sums that wrap, a request past
    the wrap counts as one that fits, and the slot map's search ends at it with a token number below
    0, hence a table column below 0."""
    new, n_new, page = [(1 << 31) - 1, 7, 5, 5], 20, 16
    first = [0]
    for n in new:
        first.append(device_int32(first[-1] + n))
    assert first[4] <= n_new  # request 3 "fits"
    lo, hi, i = 0, 3, 12
    while lo < hi:  # the last request that starts at or before slot i
        mid = (lo + hi + 1) // 2
        lo, hi = (mid, hi) if first[mid] <= i else (lo, mid - 1)
    t = device_int32(i - first[lo])
    assert lo == 3 and t < 0 and t // page < 0
    stopped = [0]
    for n in new:
        stopped.append(min(stopped[-1] + n, (1 << 31) - 1))
    assert stopped[1:] == sorted(stopped[1:]) and stopped[2] > n_new
