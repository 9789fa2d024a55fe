"""What the 8-bit products (where CTAs share a unit's K) and the norm make of a wait
that gives up, without a GPU fault: NaN, never a sum with a part missing or a row
that did not come, and the products' error word."""
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


@pytest.mark.parametrize("N,H,turn", [(64, 128, 16), (41, 136, 8), (33, 256, 8)])
def test_norm_rows_that_never_come_are_nan_in_the_residual_too(N, H, turn):
    g = torch.Generator(device="cuda").manual_seed(N)
    x, r = (torch.randn((N, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    want = binding.add_rmsnorm(x, w, r, inv_rms=True)
    got = binding.selftest_rmsnorm_wait_timeout(x, w, r.clone())
    for k in ("res", "y", "inv_rms"):
        assert torch.equal(got[k][:2 * turn], want[k][:2 * turn]), k
        assert bool(got[k][2 * turn:].isnan().all()), k
    again = binding.add_rmsnorm(x, w, r, inv_rms=True)
    assert all(torch.equal(again[k], want[k]) for k in want)
