"""Refusals of the 8-bit products' self-test entry point, without a GPU."""
import pytest

from mixture_experts_routed_non_b200 import binding

A = 1 << 20


@pytest.mark.parametrize("bad", [dict(out=None), dict(err=None), dict(out=A + 8), dict(err=A + 2), dict(us=0), dict(us=2000001)])
def test_selftest_refuses(bad):
    kw = dict(pairs=0, lose=1, out=A, err=A, us=1000, stream=None)
    assert binding.load().moe_fp8_selftest_wait_timeout(*{**kw, **bad}.values()) == binding.MOE_ERR_ARG
