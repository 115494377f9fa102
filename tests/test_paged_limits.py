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
