"""Which kernel the 8-bit products take, without a GPU: a device of 148 SMs on which 74 clusters of two
CTAs, 33 of four and 15 of eight run at once."""
import pytest

from mixture_experts_routed_non_b200 import binding


def plan(*a, **kw):
    return binding.product_plan_fp8(*a, num_sms=148, clusters=(74, 33, 15), **kw)


@pytest.mark.parametrize("P,E,K,N", [(8, 8, 4096, 1024), (8, 8, 4096, 1536), (2, 2, 8192, 512), (1, 1, 2048, 4096)])
def test_a_unit_of_the_up_product_is_256_weight_rows(P, E, K, N):
    """The few-row kernels share K out by the units there are: as many as of a product half as wide."""
    up, half = plan(P, K, N, E, swiglu=True), plan(P, K, N // 2, E)
    assert up[0] == half[0] == 32 and up[1] == half[1]


@pytest.mark.parametrize("P,E,K,N,f32,chunk", [
    # segments whose units fit one to an SM count as few rows (fp32 scales, H 7168, I 256, 8 and 16 experts of 128 and 64
    # rows: layers of 72 and 87 us in chunks, 80 and 96 in tiles)
    (1024, 8, 7168, 512, True, 32), (1024, 16, 7168, 512, True, 32),
    # and a block of their two weight tiles as twice the bytes (e8m0, 4 experts of 64 rows, H 7168, I 256: 37.6 us in
    # chunks of 32, 40.8 of 64; 4 of 32, H 1024, I 512: 26.2 in chunks of 32, 24.7 in tiles)
    (256, 4, 7168, 512, False, 32), (128, 4, 1024, 1024, False, 0),
    # few rows an expert: chunks of 32 whatever the lines say of full ones
    (32, 8, 2048, 1536, False, 32), (128, 8, 2048, 1536, False, 32)])
def test_up_product_of_few_experts(P, E, K, N, f32, chunk):
    assert plan(P, K, N, E, swiglu=True, f32=f32)[0] == chunk


@pytest.mark.parametrize("P,E,K,N,f32,want", [
    (1, 0, 7168, 4096, False, (32, 4)), (128, 0, 7168, 4096, False, (128, 4)), (512, 0, 7168, 4096, False, (0, 2)),
    (8192, 0, 7168, 4096, False, (0, 1)), (256, 0, 7168, 3584, True, (0, 4)), (1, 0, 7168, 4096, True, (32, 4)),
    (1024, 256, 512, 2048, False, (32, 1)), (4096, 128, 768, 2048, False, (64, 1)), (131072, 128, 768, 2048, False, (0, 1))])
def test_plans_of_other_products(P, E, K, N, f32, want):
    assert plan(P, K, N, E, f32=f32) == want


@pytest.mark.parametrize("bad,status", [
    (dict(P=0), "ARG"), (dict(P=1 << 31), "ARG"), (dict(E=-1), "ARG"), (dict(E=1025), "ARG"), (dict(num_sms=-1), "ARG"),
    (dict(num_sms=0, clusters=(1, 1, 1)), "ARG"), (dict(clusters=None), "ARG"), (dict(clusters=(74, 33, 256)), "ARG"),
    (dict(E=0, swiglu=True), "ARG"), (dict(K=8), "SHAPE"), (dict(K=264), "SHAPE"), (dict(N=12), "SHAPE"),
    (dict(N=264, swiglu=True), "SHAPE"), (dict(P=1 << 30, N=1 << 24), "SHAPE")])
def test_plan_refuses(bad, status):
    kw = dict(P=4, K=256, N=256, E=2, num_sms=148, clusters=(74, 33, 15))
    kw.update(bad)
    with pytest.raises(binding.MoeError) as e:
        binding.product_plan_fp8(kw.pop("P"), kw.pop("K"), kw.pop("N"), kw.pop("E"), **kw)
    assert e.value.status == getattr(binding, "MOE_ERR_" + status)
