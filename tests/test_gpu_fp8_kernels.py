"""Every kernel, chunk and split of K that the products of segments take, on the GPU against the 64-bit
definitions; each case asserts which one it reaches (moe_fp8_product_plan)."""
import pytest
import torch

import fp8_ref as ref
from mixture_experts_routed_non_b200 import binding
from test_gpu_fp8 import BF16, E8, F32, _grouped_case, _grouped_ref, _layer_case, _layer_ref

pytestmark = pytest.mark.gpu

MANY = [20 + (7 * e) % 29 for e in range(64)]  # 20 to 48 rows each: partial chunks of 64

# rows of each segment, K, N -> the kernel with e8m0 scales, with fp32 ones: (rows to a chunk or 0 for pairs, split of K)
GROUPED = {
    "chunks_of_64": (MANY, 384, 520, (64, 1), (0, 1)),
    "split_2": ([5, 0, 9, 1], 1024, 520, (32, 2), (32, 2)),
    "split_4": ([5, 0, 9, 32], 2064, 264, (32, 4), (32, 4)),
    "split_8": ([5, 0, 9], 4112, 264, (32, 8), (32, 8)),
    "split_2_full_chunks": ([60, 64, 50], 2064, 1032, (32, 2), (32, 2)),
    "split_8_full_chunks": ([60, 64], 4112, 264, (32, 8), (32, 8)),
    "chunks_of_64_split_2": ([130, 0, 117], 4112, 1160, (64, 2), (32, 1)),
}


@pytest.mark.parametrize("name", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("scale", [E8, F32])
def test_grouped(name, gather, scale):
    counts, K, N, e8m0, f32 = GROUPED[name]
    want = e8m0 if scale == E8 else f32
    a, s, off, w, t, b, idx, P = _grouped_case(counts, K, N, gather, scale, scale, True, len(name), spare=3)
    plan = binding.product_plan_fp8(P, K, N, len(counts), f32=scale == F32)
    assert plan == want
    out = torch.full((P, N), 77.0, dtype=BF16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.grouped_linear_fp8(a, s, off, w, t, b, gather=idx, out=out, err=err)
    y, tol = _grouped_ref(counts, a, s, w, t, b, idx)
    ref.check(out[:P - 3], y, tol, name)
    assert bool((out[P - 3:] == 77).all()) and int(err) == 0
    for _ in range(3):  # the parts of K are added in a fixed order
        assert torch.equal(binding.grouped_linear_fp8(a, s, off, w, t, b, gather=idx)[:P - 3], out[:P - 3])


# N, H, I, E, top k -> up and down with e8m0 scales, with fp32 ones
LAYERS = {
    "chunks_of_64": ((512, 512, 256, 64, 4), ((64, 1), (64, 1)), ((32, 1), (32, 1))),
    "chunks_of_64_odd": ((700, 384, 384, 80, 4), ((64, 1), (64, 1)), ((0, 1), (0, 1))),
    "split_2_2": ((3, 1024, 1024, 4, 2), ((32, 2), (32, 2)), ((32, 2), (32, 2))),
    "split_4_2": ((6, 2048, 1024, 4, 2), ((32, 4), (32, 2)), ((32, 4), (32, 2))),
    "split_8_up": ((5, 4096, 512, 2, 2), ((32, 8), (32, 1)), ((32, 8), (32, 1))),
    "split_8_up_full_chunks": ((60, 4096, 128, 2, 1), ((32, 8), (32, 1)), ((32, 8), (32, 1))),
    "split_8_down": ((60, 256, 4096, 2, 1), ((32, 1), (32, 8)), ((32, 1), (32, 8))),
    "chunks_of_64_split_4": ((120, 2048, 1024, 2, 1), ((64, 4), (32, 1)), ((32, 2), (32, 1))),
}


@pytest.mark.parametrize("name", LAYERS)
@pytest.mark.parametrize("layout", [binding.LAYOUT_INTERLEAVED, binding.LAYOUT_CONCATENATED])
@pytest.mark.parametrize("scale", [E8, F32])
def test_layer(name, layout, scale):
    (N, H, I, E, K), e8m0, f32 = LAYERS[name]
    plans = (binding.product_plan_fp8(N * K, H, 2 * I, E, swiglu=True, f32=scale == F32),
             binding.product_plan_fp8(N * K, I, H, E, f32=scale == F32))
    assert plans == (e8m0 if scale == E8 else f32)
    c = _layer_case(N, H, I, E, K, 0.0, True, scale, scale, 3 + layout)
    y, tol = _layer_ref(*c, layout)
    out = binding.forward_fp8(*c, layout=layout)
    ref.check(out, y, tol, name)
    assert torch.equal(out, binding.forward_fp8(*c, layout=layout))
