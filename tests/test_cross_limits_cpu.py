"""Limits of pa_cross_attention that are checked before any CUDA call, on a machine without a GPU."""
import pytest

from paged_kv_cache_456_b200 import ops

from tests.test_cross_cpu import call, lib  # noqa: F401  (a fixture)


@pytest.mark.parametrize("dt", [ops.PA_BF16, ops.PA_F32])
def test_contexts_longer_than_fp32_sums_can_hold(lib, dt):  # noqa: F811
    longest = 1 << 24
    for blocks, max_len in ((longest // 16 + 1, longest + 1), (1 << 26, 1 << 30), (1 << 22, (1 << 31) - 1)):
        assert call(lib, B=blocks, max_len=max_len, dt=dt) == ops.PA_ERR_UNSUPPORTED
    # the longest is taken (what it meets next is the missing device or the small workspace)
    for blocks, max_len in ((longest // 16, longest), (longest // 16, 1 << 30), (1 << 26, longest)):
        assert call(lib, B=blocks, max_len=max_len, dt=dt, bytes=16) not in (ops.PA_OK, ops.PA_ERR_UNSUPPORTED)
