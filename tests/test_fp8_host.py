"""Refusals of the norm, the quantisers and the 8-bit products, without a GPU:
the C entry points with fake, never-dereferenced addresses, and the binding's
tensor checks on CPU tensors.  And the norm's gradient formula against
differences."""
import ctypes

import pytest
import torch

import fp8_ref as ref
from mixture_experts_routed_non_b200 import binding

A = 1 << 20
ARG, SHAPE, WS = binding.MOE_ERR_ARG, binding.MOE_ERR_SHAPE, binding.MOE_ERR_WS
NO_DEVICE = (binding.MOE_ERR_CUDA, binding.MOE_ERR_DEVICE)
E4, E8, BF = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def _call(fn, defaults, **kw):
    assert set(kw) <= set(defaults), kw
    st = fn(*{**defaults, **kw}.values())
    return st


NORM = dict(x=A, residual=A, weight=A, N=4, H=256, eps=1e-6, res=A, y=A, y8=A, y8_scale=A, inv_rms=A, stream=None)
BACK = dict(dy=A, res=A, weight=A, inv_rms=A, dres=A, N=4, H=256, dx=A, dweight=A, ws=A, ws_bytes=1 << 30, stream=None)
ROWS = dict(x=A, M=4, K=256, q=A, scale=A, stream=None)
WEIGHT = dict(w=A, E=2, K=256, N=128, q=A, scale=A, stream=None)
LINEAR = dict(a=A, a_scale=A, a_sd=0, M=4, K=256, w=A, w_scale=A, w_sd=0, N=128, bias=A, out=A, err=A, stream=None)
GROUPED = dict(a=A, a_scale=A, a_sd=0, rows=4, K=256, gather=None, P=4, off=A, E=2, w=A, w_scale=A, w_sd=0, N=128,
               bias=A, out=A, err=A, stream=None)


@pytest.mark.parametrize("name,defaults,bad,status", [
    ("moe_add_rmsnorm", NORM, bad, st) for bad, st in [
        (dict(x=None), ARG), (dict(weight=None), ARG), (dict(N=-1), ARG), (dict(N=1 << 31), ARG), (dict(H=0), SHAPE),
        (dict(H=12), SHAPE), (dict(H=16392), SHAPE), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
        (dict(residual=None), ARG), (dict(res=None), ARG), (dict(y8=None), ARG), (dict(y8_scale=None), ARG),
        (dict(y=None, y8=None, y8_scale=None), ARG), (dict(x=A + 8), ARG), (dict(residual=A + 2), ARG),
        (dict(weight=A + 4), ARG), (dict(y=A + 8), ARG), (dict(y8=A + 8), ARG), (dict(inv_rms=A + 2), ARG)]
] + [
    ("moe_add_rmsnorm_backward", BACK, bad, st) for bad, st in [
        (dict(dy=None), ARG), (dict(res=None), ARG), (dict(weight=None), ARG), (dict(inv_rms=None), ARG),
        (dict(dx=None), ARG), (dict(dweight=None), ARG), (dict(H=20), SHAPE), (dict(H=1 << 20), SHAPE), (dict(N=-2), ARG),
        (dict(dres=A + 8), ARG), (dict(dx=A + 2), ARG), (dict(dweight=A + 1), ARG), (dict(ws=None), WS),
        (dict(ws=A + 16), WS), (dict(ws_bytes=255), WS)]
] + [
    ("moe_fp8_quantize_rows", ROWS, bad, st) for bad, st in [
        (dict(x=None), ARG), (dict(q=None), ARG), (dict(scale=None), ARG), (dict(M=-1), ARG), (dict(K=8), SHAPE),
        (dict(K=24), SHAPE), (dict(x=A + 2), ARG), (dict(q=A + 8), ARG), (dict(M=1 << 30, K=1 << 28), SHAPE)]
] + [
    ("moe_fp8_quantize_weight", WEIGHT, bad, st) for bad, st in [
        (dict(w=None), ARG), (dict(q=None), ARG), (dict(scale=None), ARG), (dict(E=0), ARG), (dict(E=1025), ARG),
        (dict(K=40), SHAPE), (dict(N=4), SHAPE), (dict(N=65535 * 128 + 8), SHAPE), (dict(w=A + 2), ARG)]
] + [
    ("moe_fp8_linear", LINEAR, bad, st) for bad, st in [
        (dict(a=None), ARG), (dict(a_scale=None), ARG), (dict(w=None), ARG), (dict(w_scale=None), ARG), (dict(out=None), ARG),
        (dict(M=-1), ARG), (dict(M=1 << 31), ARG), (dict(K=0), SHAPE), (dict(K=136), SHAPE), (dict(N=0), SHAPE),
        (dict(N=12), SHAPE), (dict(a_sd=2), ARG), (dict(w_sd=-1), ARG), (dict(a=A + 8), ARG), (dict(w=A + 8), ARG),
        (dict(out=A + 2), ARG), (dict(bias=A + 1), ARG), (dict(err=A + 2), ARG), (dict(a_sd=1, a_scale=A + 2), ARG),
        (dict(w_sd=1, w_scale=A + 1), ARG), (dict(K=1 << 20, N=1 << 20), SHAPE), (dict(M=1 << 30, N=1 << 24), SHAPE)]
] + [
    ("moe_fp8_grouped_linear", GROUPED, bad, st) for bad, st in [
        (dict(off=None), ARG), (dict(off=A + 2), ARG), (dict(E=0), ARG), (dict(E=1025), ARG), (dict(P=5), ARG),
        (dict(gather=A + 2), ARG), (dict(gather=A, rows=0), ARG), (dict(rows=-1), ARG), (dict(gather=A, P=-1), ARG)]
])
def test_c_entry_points_refuse(lib, name, defaults, bad, status):
    assert _call(getattr(lib, name), defaults, **bad) == status


@pytest.mark.parametrize("name,defaults", [("moe_add_rmsnorm", NORM), ("moe_add_rmsnorm_backward", BACK),
                                           ("moe_fp8_quantize_rows", ROWS), ("moe_fp8_quantize_weight", WEIGHT),
                                           ("moe_fp8_linear", LINEAR), ("moe_fp8_grouped_linear", GROUPED)])
def test_good_arguments_reach_the_device_query(lib, name, defaults):
    if torch.cuda.is_available():
        pytest.skip("a device is present: the fake addresses must not reach a kernel")
    assert _call(getattr(lib, name), defaults) in NO_DEVICE


def _layer_args(**kw):
    r = binding.MoeRouting()
    r.kind, r.index_dtype, r.N, r.K, r.pairs = binding.ROUTING_TOPK, binding.INDEX_INT32, 8, 2, -1
    r.expert_idx = r.weights = A
    r.token_idx = None
    d = dict(x=A, xs=A, xsd=0, r=ctypes.byref(r), H=256, I=128, E=4, w1=A, s1=A, sd1=0, b1=None, w2=A, s2=A, sd2=0,
             b2=None, act=0, lay=0, out=A, meta=None, ws=A, wsb=1 << 30, stream=None)
    d.update(kw)
    return tuple(d.values())


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), ARG), (dict(xs=None), ARG), (dict(w1=None), ARG), (dict(s1=None), ARG), (dict(w2=None), ARG),
    (dict(s2=None), ARG), (dict(out=None), ARG), (dict(xsd=3), ARG), (dict(sd1=2), ARG), (dict(sd2=-1), ARG),
    (dict(act=1), ARG), (dict(lay=2), ARG), (dict(H=192), SHAPE), (dict(I=64), SHAPE), (dict(H=0), SHAPE),
    (dict(x=A + 8), ARG), (dict(w2=A + 4), ARG), (dict(sd1=1, s1=A + 2), ARG), (dict(b1=A + 1), ARG), (dict(ws=None), WS),
    (dict(ws=A + 128), WS), (dict(wsb=1000), WS), (dict(E=0), ARG), (dict(r=None), ARG), (dict(H=1 << 26, I=1 << 26), SHAPE)])
def test_layer_refuses(lib, bad, status):
    assert lib.moe_fp8_forward(*_layer_args(**bad)) == status


def test_workspace_sizes(lib):
    n = lib.moe_add_rmsnorm_backward_workspace_bytes(4, 256)
    assert n >= 256 * 4
    assert _call(lib.moe_add_rmsnorm_backward, BACK, ws_bytes=n - 1) == WS
    assert lib.moe_add_rmsnorm_backward_workspace_bytes(0, 256) > 0
    assert lib.moe_add_rmsnorm_backward_workspace_bytes(4, 12) == 0
    with pytest.raises(binding.MoeError):
        binding.add_rmsnorm_backward_workspace_bytes(4, 12)
    idx, w = torch.zeros((8, 2), dtype=torch.int32), torch.zeros((8, 2))
    r = binding.routing(idx, w)
    # the 8-bit workspace holds h in half the bytes of the bf16 one and no training buffers
    assert 0 < binding.fp8_workspace_bytes(r, 256, 128, 4) <= binding.routed_workspace_bytes(r, 256, 128, 4) + 8192
    with pytest.raises(binding.MoeError):
        binding.fp8_workspace_bytes(r, 192, 128, 4)


def _cpu():
    x = torch.zeros((4, 256), dtype=BF)
    a, s = x.to(E4), torch.ones((4, 2)).to(E8)
    w, t = torch.zeros((128, 256)).to(E4), torch.ones((1, 2)).to(E8)
    return x, torch.ones(256, dtype=BF), a, s, w, t


def test_binding_refuses_bad_tensors():
    x, nw, a, s, w, t = _cpu()
    n, bk, lin, grp = binding.add_rmsnorm, binding.add_rmsnorm_backward, binding.linear_fp8, binding.grouped_linear_fp8
    inv, off = torch.ones(4), torch.tensor([0, 2, 4], dtype=torch.int32)
    w3, t3 = w[None].repeat(2, 1, 1), t.float()[None].repeat(2, 1, 1)
    type_errors = [
        lambda: n(x.float(), nw), lambda: n(x, nw.float()), lambda: n(x, nw, x.half()), lambda: lin(x, s, w, t),
        lambda: lin(a, s.view(torch.uint8), w, t), lambda: lin(a, s.float().half(), w, t), lambda: lin(a, s, w, t, nw.float()),
        lambda: grp(a, s, off.long(), w3, t3), lambda: grp(a, s, off, w3, t3, gather=off.long()),
        lambda: bk(x, x, nw, inv.double()), lambda: binding.quantize_rows_fp8(x.float()),
        lambda: binding.quantize_weight_fp8(x.half()), lambda: n(x, nw, out=dict(y=x.float())),
    ]
    value_errors = [
        lambda: n(x[0], nw), lambda: n(x, nw[:8]), lambda: n(x[:, ::2], nw[::2]), lambda: n(x.t(), nw[:4]), lambda: n(x, nw, x[:3]),
        lambda: n(x, nw, y=False), lambda: n(x, nw, out=dict(res=x)), lambda: n(x, nw, out=dict(z=x)),
        lambda: lin(a, s[:, :1], w, t), lambda: lin(a, s, w[:, :128], t), lambda: lin(a, s, w, t.float().repeat(2, 1)),
        lambda: lin(a, s, w, t, nw[:64]), lambda: lin(a.t(), s, w, t), lambda: lin(a, s, w3, t3), lambda: lin(a, s, w, t, out=x),
        lambda: grp(a, s, off[:2], w3, t3), lambda: grp(a, s, off, w, t), lambda: grp(a, s, off, w3, t3[:1]),
        lambda: bk(x, x, nw, inv[:3]), lambda: bk(x, x[:2], nw, inv), lambda: bk(x, x, nw, inv, dres=x[:, :8]),
        lambda: binding.quantize_weight_fp8(x[0]),
        # sound arguments, but not on a GPU
        lambda: n(x, nw), lambda: lin(a, s, w, t), lambda: grp(a, s, off, w3, t3), lambda: bk(x, x, nw, inv),
        lambda: binding.quantize_rows_fp8(x), lambda: binding.quantize_weight_fp8(x),
    ]
    for f in type_errors:
        with pytest.raises(TypeError):
            f()
    for i, f in enumerate(value_errors):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")


def test_layer_binding_refuses_bad_tensors():
    x, _, a, s, _, _ = _cpu()
    idx, tw = torch.zeros((4, 2), dtype=torch.int32), torch.ones((4, 2))
    w1, s1 = torch.zeros((3, 256, 256)).to(E4), torch.ones((3, 2, 2))
    w2, s2 = torch.zeros((3, 256, 128)).to(E4), torch.ones((3, 2, 1))
    f = binding.forward_fp8
    with pytest.raises(TypeError):
        f(x, s, idx, tw, w1, s1, w2, s2)
    with pytest.raises(TypeError):
        f(a, s, idx.float(), tw, w1, s1, w2, s2)
    for bad in [lambda: f(a, s[:3], idx, tw, w1, s1, w2, s2), lambda: f(a, s, idx, tw, w1, s1[:, :1], w2, s2),
                lambda: f(a, s, idx, tw, w1, s1, w2[:, :128], s2), lambda: f(a, s, idx[:3], tw[:3], w1, s1, w2, s2),
                lambda: f(a, s, idx, tw, w1, s1, w2, s2, torch.zeros((3, 128), dtype=BF)),
                lambda: f(a, s, idx, tw, w1, s1, w2, s2)]:
        with pytest.raises(ValueError):
            bad()


def test_gradient_formula_against_differences():
    """The 64-bit formula the GPU test uses, against central differences of the 64-bit norm."""
    g = torch.Generator().manual_seed(1)
    N, H, eps = 3, 24, 1e-3
    s = torch.randn((N, H), generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn((H,), generator=g, dtype=torch.float64)
    dy = torch.randn((N, H), generator=g, dtype=torch.float64)
    dres = torch.randn((N, H), generator=g, dtype=torch.float64)
    inv_of = lambda v: 1 / torch.sqrt(v.square().mean(-1) + eps)
    loss = lambda v, u: (dy * v * inv_of(v)[:, None] * u).sum() + (dres * v).sum()
    dx, dw = ref.norm_backward(dy, s, w, inv_of(s), dres)
    h = 1e-6
    for t in range(N):
        for j in range(H):
            d = torch.zeros_like(s)
            d[t, j] = h
            # central difference: error O(h^2) ~ 1e-12 and 1e-16 / h ~ 1e-10 of rounding
            assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * h) - dx[t, j]) < 1e-7
    for j in range(H):
        d = torch.zeros_like(w)
        d[j] = h
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * h) - dw[j]) < 1e-7


def test_scale_and_rounding_of_the_reference():
    """round_e4m3 against torch's conversion on every code and the midpoints between codes."""
    codes = torch.arange(0, 0x7F, dtype=torch.uint8).view(E4).float().double()
    mids = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mids, mids * (1 + 2.0 ** -20), mids * (1 - 2.0 ** -20)])
    v = torch.cat([v, -v])
    assert torch.equal(ref.round_e4m3(v), v.float().to(E4).float().double())
    amax = torch.tensor([0.0, 448.0, 448.0001, 224.0, 1.75, 1.7501, 2.0 ** -140], dtype=torch.float64)
    assert ref.pow2_scale(amax).tolist() == [1.0, 1.0, 2.0, 0.5, 2.0 ** -8, 2.0 ** -7, 2.0 ** -126]


def _big(shape, dtype):
    """A tensor that has a shape but no memory."""
    return torch.empty(shape, dtype=dtype, device="meta")


def test_binding_refuses_sizes_past_32_bits():
    """A size that the C entry point takes as int32 is refused, not cut to its low bits (2^32 + 256 -> 256)."""
    b = (1 << 32) + 256
    e, f32 = b // 128, torch.float32
    idx, tw = torch.zeros((4, 2), dtype=torch.int32), torch.ones((4, 2))
    r = binding.routing(idx, tw)
    calls = [
        lambda: binding.add_rmsnorm(_big((1, b), BF), _big((b,), BF)),
        lambda: binding.add_rmsnorm_backward(_big((1, b), BF), _big((1, b), BF), _big((b,), BF), _big((1,), f32)),
        lambda: binding.add_rmsnorm_backward_workspace_bytes(4, b),
        lambda: binding.quantize_rows_fp8(_big((1, b), BF)),
        lambda: binding.quantize_weight_fp8(_big((b, 16), BF)),
        lambda: binding.quantize_weight_fp8(_big((2, 16, b), BF)),
        lambda: binding.quantize_weight_fp8(_big((b, 16, 8), BF)),
        lambda: binding.linear_fp8(_big((1, b), E4), _big((1, e), E8), _big((8, b), E4), _big((1, e), E8)),
        lambda: binding.linear_fp8(_big((1, 16), E4), _big((1, 1), E8), _big((b, 16), E4), _big((e, 1), E8)),
        lambda: binding.grouped_linear_fp8(_big((1, b), E4), _big((1, e), E8), _big((2,), torch.int32), _big((1, 8, b), E4),
                                           _big((1, 1, e), E8)),
        lambda: binding.grouped_linear_fp8(_big((1, 16), E4), _big((1, 1), E8), _big((b + 1,), torch.int32),
                                           _big((b, 8, 16), E4), _big((b, 1, 1), E8)),
        lambda: binding.forward_fp8(_big((4, b), E4), _big((4, e), E8), idx, tw, _big((2, 256, b), E4), _big((2, 2, e), E8),
                                    _big((2, b, 128), E4), _big((2, e, 1), E8)),
        lambda: binding.fp8_workspace_bytes(r, 256, b, 4),
        lambda: binding.product_plan_fp8(4, b, 256, num_sms=148, clusters=(74, 33, 15)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(binding.MoeError) as err:
            call()
            pytest.fail(f"call {i} was accepted")
        assert err.value.status == SHAPE, i


def test_norm_refuses_y_and_res_in_one_buffer():
    """res may be x, and y may be x, but the second to be written would replace the first."""
    x, w, r = torch.zeros((4, 256), dtype=BF), torch.ones(256, dtype=BF), torch.zeros((4, 256), dtype=BF)
    with pytest.raises(ValueError, match="same buffer"):
        binding.add_rmsnorm(x, w, r, out=dict(res=x, y=x))


def test_message_of_a_bad_shape_names_the_bf16_multiple():
    assert "multiples of 64" in binding.strerror(SHAPE)
