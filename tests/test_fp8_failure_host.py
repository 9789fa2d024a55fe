"""Refusals of the self-test entry points of the 8-bit products and the norm, without a GPU."""
import pytest

from mixture_experts_routed_non_b200 import binding

A = 1 << 20


@pytest.mark.parametrize("bad", [dict(out=None), dict(err=None), dict(out=A + 8), dict(err=A + 2), dict(us=0), dict(us=2000001)])
def test_selftest_refuses(bad):
    kw = dict(pairs=0, lose=1, out=A, err=A, us=1000, stream=None)
    assert binding.load().moe_fp8_selftest_wait_timeout(*{**kw, **bad}.values()) == binding.MOE_ERR_ARG


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), "ARG"), (dict(residual=None), "ARG"), (dict(res=None), "ARG"), (dict(y=None), "ARG"), (dict(N=0), "ARG"),
    (dict(N=4097), "ARG"), (dict(H=264), "SHAPE"), (dict(H=12), "SHAPE")])
def test_norm_selftest_refuses(bad, status):
    kw = dict(x=A, residual=A, weight=A, N=4, H=128, eps=1e-6, res=A, y=A, inv_rms=A, stream=None)
    st = binding.load().moe_add_rmsnorm_selftest_wait_timeout(*{**kw, **bad}.values())
    assert st == getattr(binding, "MOE_ERR_" + status)
