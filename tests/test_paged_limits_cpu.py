"""Sizes that the kernels' 32-bit counters do not hold are refused by the C ABI, on the CPU."""
import pytest

from long_sequence_context_b200 import cpattn as cp
from tests.test_paged_cpu import VP, _c_decode


def _plan(R):
    return cp.lib.cpattn_cache_plan(VP, VP, VP, R, 1, 16, VP, VP, 16, VP, VP, VP, VP, 4, VP, VP, 1 << 40, None)


def test_plan_requests():
    """Its search halves sums of two request numbers: up to 2^30 requests."""
    n0 = cp.launch_count()
    for R in ((1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1):
        assert _plan(R) == cp.ERR_SHAPE
    assert cp.launch_count() == n0


def test_append_heads():
    """A block counts the heads of up to 32 stretches of tokens as an int: up to 2^25 heads."""
    n0 = cp.launch_count()
    for heads in ((1 << 25) + 1, 1 << 26, (1 << 31) - 1):
        st = cp.lib.cpattn_cache_append(VP, VP, 64, 64, 64, 64, VP, 4, VP, VP, None, heads, 64, 16, 1, None, 0, 0, None)
        assert st == cp.ERR_SHAPE
    assert cp.launch_count() == n0


@pytest.mark.parametrize("Hq,Hkv,D", [((1 << 23) + 64, (1 << 17) + 1, 128), (1 << 25, 1 << 19, 64), (1 << 26, 1 << 26, 128)])
def test_decode_outputs_of_a_request(Hq, Hkv, D):
    """The outputs of a request without a key are counted as an int: Hq * D up to 2^30."""
    n0 = cp.launch_count()
    assert _c_decode(R=1, Hq=Hq, Hkv=Hkv, D=D, width=1, pages=1) == cp.ERR_SHAPE
    assert cp.launch_count() == n0
