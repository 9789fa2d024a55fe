"""What the 8-bit products make of a wait that gives up where CTAs share a unit's
K, without a GPU fault: NaN, never a sum with a part missing, and the error word."""
import pytest
import torch

from mixture_experts_routed_non_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [False, True])
def test_shared_sums_are_whole(pairs):
    out, err = binding.selftest_fp8_wait_timeout(pairs, False, 500000)
    assert int(err) == 0 and bool((out == 3).all())


@pytest.mark.parametrize("pairs", [False, True])
def test_a_part_that_never_comes_makes_nan(pairs):
    out, err = binding.selftest_fp8_wait_timeout(pairs, True, 20000)  # 20 ms
    assert int(err) == binding.DEVERR_TIMEOUT
    assert bool(out.isnan().all())
    test_shared_sums_are_whole(pairs)  # the context and the next call are as before
