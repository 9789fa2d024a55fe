"""RMS norm with the residual's addition (bf16 and 8-bit outputs), its gradient,
and the two quantisers, on the GPU against their 64-bit definitions."""
import pytest
import torch

import fp8_ref as ref
from mixture_experts_routed_non_b200 import binding

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
# one thread's columns, one warp's, whole blocks, a block's end inside, the widest row
SIZES = [(1, 8), (1, 2048), (3, 136), (37, 1000), (129, 2048), (5, 7168), (2, 16384), (300, 128), (64, 1032), (7, 4104)]
FP32 = 2.0 ** -18  # 64 fp32 roundings: sums of up to 16384 squares in a tree of at most 64 steps


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _inputs(N, H, seed):
    g = _gen(seed)
    x = torch.randn((N, H), generator=g, device="cuda").to(BF16)
    r = (3 * torch.randn((N, H), generator=g, device="cuda")).to(BF16)
    w = (1 + 0.3 * torch.randn((H,), generator=g, device="cuda")).to(BF16)
    return x, r, w


def _check_forward(out, x, residual, w, eps):
    s, inv, y = ref.norm(x, residual, w, eps)
    if residual is not None:
        assert torch.equal(out["res"].double(), s)
    if "inv_rms" in out:
        ref.check(out["inv_rms"], inv, FP32 * inv, "inv_rms")
    if "y" in out:
        ref.check(out["y"], y, (2.0 ** -8 + 2 * FP32) * y.abs() + 2.0 ** -133, "y")
    if "y8" in out:
        sc = out["y8_scale"].float().double()
        amax = ref.to_blocks(y).abs().amax(-1)
        nz = amax > 0
        assert torch.equal(torch.frexp(sc)[0], torch.full_like(sc, 0.5))          # powers of two
        assert bool((amax <= 448 * sc * (1 + 2 * FP32))[nz].all())                # the smallest that holds amax
        assert bool((amax > 224 * sc * (1 - 2 * FP32))[nz].all())
        assert bool((sc == 1)[~nz].all())
        v = ref.values(out["y8"], out["y8_scale"])
        step = sc.repeat_interleave(128, -1)[:, :y.shape[1]]
        ref.check(v, y, 2.0 ** -4 * (1 + FP32) * y.abs() + 2.0 ** -10 * step + FP32 * y.abs(), "y8")


@pytest.mark.parametrize("N,H", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(N, H, residual):
    x, r, w = _inputs(N, H, N * 7 + H)
    r = r if residual else None
    for kw in (dict(y=True, fp8=True, inv_rms=True), dict(y=False, fp8=True), dict(y=True, inv_rms=True), dict()):
        out = binding.add_rmsnorm(x, w, r, eps=1e-5, **kw)
        assert set(out) == ({"res"} if residual else set()) | {k for k, v in dict(
            y=kw.get("y", True), y8=kw.get("fp8"), y8_scale=kw.get("fp8"), inv_rms=kw.get("inv_rms")).items() if v}
        _check_forward(out, x, r, w, 1e-5)


def test_norm_outputs_agree_whatever_else_is_asked():
    x, r, w = _inputs(61, 2056, 3)
    full = binding.add_rmsnorm(x, w, r, y=True, fp8=True, inv_rms=True)
    a = binding.add_rmsnorm(x, w, r)
    b = binding.add_rmsnorm(x, w, r, y=False, fp8=True)
    assert torch.equal(full["y"], a["y"]) and torch.equal(full["res"], b["res"])
    assert torch.equal(full["y8"].view(torch.uint8), b["y8"].view(torch.uint8))
    assert torch.equal(full["y8_scale"].view(torch.uint8), b["y8_scale"].view(torch.uint8))


def test_norm_in_place_and_given_buffers():
    x, r, w = _inputs(33, 2048, 4)
    want = binding.add_rmsnorm(x, w, r, fp8=True, inv_rms=True)
    r2, x2 = r.clone(), x.clone()
    buf = dict(res=r2, y=x2, inv_rms=torch.full((33,), 7.0, device="cuda"))  # res over residual, y over x
    got = binding.add_rmsnorm(x2, w, r2, fp8=True, inv_rms=True, out=buf)
    assert got["res"] is r2 and got["y"] is x2
    for k in want:
        assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k


def test_norm_zero_tiny_and_huge_rows():
    x, _, w = _inputs(6, 384, 5)
    x[0] = 0
    x[1, :128] = 0                      # one block of zeros in a row that is not
    x[2] = x[2] * 2.0 ** -60            # eps decides
    x[3] = x[3] * 2.0 ** 50
    x[4] = 0
    x[4, 200] = -2.0
    out = binding.add_rmsnorm(x, w, None, eps=1e-6, fp8=True, inv_rms=True)
    _check_forward(out, x, None, w, 1e-6)
    assert bool((out["y"][0] == 0).all()) and bool((out["y8_scale"][0].float() == 1).all())


def test_norm_nonfinite_rows():
    x, _, w = _inputs(4, 512, 6)
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    out = binding.add_rmsnorm(x, w, None, fp8=True)
    for row in (0, 3):  # the others are untouched by it
        _check_forward({k: v[row:row + 1] for k, v in out.items()}, x[row:row + 1], None, w, 1e-6)
    assert bool(out["y"][1].isnan().all()) and bool(out["y8"][1].float().isnan().all())
    # an infinity makes 1/rms 0: its own place is NaN, the others 0
    nan = torch.zeros(512, dtype=torch.bool, device="cuda")
    nan[300] = True
    assert torch.equal(out["y"][2].isnan(), nan) and torch.equal(out["y8"][2].float().isnan(), nan)
    assert bool((out["y"][2][~nan] == 0).all())
    assert bool((out["y8_scale"][1:3].float() == 1).all())


def test_norm_no_rows():
    x = torch.empty((0, 256), dtype=BF16, device="cuda")
    w = torch.ones(256, dtype=BF16, device="cuda")
    out = binding.add_rmsnorm(x, w, x, fp8=True, inv_rms=True)
    assert out["y8"].shape == (0, 256) and out["inv_rms"].shape == (0,)
    g = binding.add_rmsnorm_backward(x, x, w, out["inv_rms"], grads=dict(dweight=torch.full((256,), 9.0, device="cuda")))
    assert g["dx"].shape == (0, 256) and bool((g["dweight"] == 0).all())


@pytest.mark.parametrize("N,H", SIZES + [(1300, 264)])
@pytest.mark.parametrize("with_dres", [False, True])
def test_norm_backward(N, H, with_dres):
    x, r, w = _inputs(N, H, N + H)
    g = _gen(N * 3 + H)
    dy = torch.randn((N, H), generator=g, device="cuda").to(BF16)
    dres = torch.randn((N, H), generator=g, device="cuda").to(BF16) if with_dres else None
    f = binding.add_rmsnorm(x, w, r, inv_rms=True)
    got = binding.add_rmsnorm_backward(dy, f["res"], w, f["inv_rms"], dres=dres)
    s, inv = f["res"].double(), f["inv_rms"].double()
    d, wd = dy.double(), w.double()
    dx, dw = ref.norm_backward(d, s, wd, inv, None if dres is None else dres.double())
    # fp32 terms: the products and the row sum of |w dy s|, each within FP32 of its magnitude
    mag = (inv[:, None] * wd * d).abs() + inv[:, None] ** 3 * (d * wd * s).abs().mean(-1, keepdim=True) * s.abs()
    if dres is not None:
        mag = mag + dres.double().abs()
    ref.check(got["dx"], dx, 2.0 ** -8 * dx.abs() + 2 * FP32 * mag + 2.0 ** -133, "dx")
    # at most N / 592 + 1 rows in a block, then a tree: fewer than 128 fp32 roundings
    ref.check(got["dweight"], dw, 2.0 ** -17 * (d * s * inv[:, None]).abs().sum(0) + 2.0 ** -140, "dweight")


def test_norm_backward_in_place_and_repeatable():
    N, H = 700, 2048
    x, r, w = _inputs(N, H, 8)
    dy, dres = _inputs(N, H, 9)[:2]
    f = binding.add_rmsnorm(x, w, r, inv_rms=True)
    a = binding.add_rmsnorm_backward(dy, f["res"], w, f["inv_rms"], dres=dres)
    ws = torch.empty(binding.add_rmsnorm_backward_workspace_bytes(N, H), dtype=torch.uint8, device="cuda").fill_(255)
    over = dy.clone()
    b = binding.add_rmsnorm_backward(over, f["res"], w, f["inv_rms"], dres=dres, grads=dict(dx=over), ws=ws)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])  # fixed order, bit for bit


@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (50, 2000), (7, 7168), (513, 256)])
def test_quantize_rows_is_the_definition(M, K):
    x = _inputs(M, K, M + K)[0]
    x[0, :16] = 0
    if M > 2:
        x[1, 3], x[1, 9], x[2, 11] = float("inf"), float("-inf"), float("nan")
        x[2, 0] = 1e30
        x[0, :128] = x[0, :128] * 2.0 ** -130  # below the smallest scale's range
    q, s = binding.quantize_rows_fp8(x)
    want, ws = ref.quantize(x.double())
    assert torch.equal(s.float().double(), ws)
    assert torch.equal(q.float().double().nan_to_num(1e9), want.nan_to_num(1e9))


@pytest.mark.parametrize("E,K,N", [(1, 16, 8), (2, 128, 128), (3, 144, 72), (2, 2000, 264), (1, 256, 1544)])
def test_quantize_weight_is_the_definition(E, K, N):
    w = (torch.randn((E, K, N), generator=_gen(E + K + N), device="cuda") / K ** 0.5).to(BF16)
    w[0, 0, 0] = float("inf")
    q, s = binding.quantize_weight_fp8(w)
    assert q.shape == (E, N, K) and s.shape == (E, ref.blocks(N), ref.blocks(K))
    t = w.double().transpose(1, 2)
    p = torch.zeros((E, ref.blocks(N) * 128, ref.blocks(K) * 128), dtype=torch.float64, device="cuda")
    p[:, :N, :K] = t
    p = p.view(E, ref.blocks(N), 128, ref.blocks(K), 128)
    sc = ref.pow2_scale(torch.where(p.isfinite(), p.abs(), torch.zeros_like(p)).amax((2, 4)))
    assert torch.equal(s.float().double(), sc)
    want = ref.round_e4m3((p / sc[:, :, None, :, None]).reshape(E, ref.blocks(N) * 128, -1)[:, :N, :K])
    assert torch.equal(q.float().double().nan_to_num(1e9), want.nan_to_num(1e9))
    if E == 1:
        q2, s2 = binding.quantize_weight_fp8(w[0])
        assert q2.shape == (N, K) and torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8))


def test_norm_of_values_whose_scale_and_rms_multiply_past_the_range():
    """1 / rms = 2^62 and a block's scale 2^-86: their quotient is no fp32 number."""
    g = _gen(9)
    sign = torch.where(torch.rand((5, 640), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x = (sign * 2.0 ** -62).to(BF16)
    w = torch.full((640,), 2.0 ** -78, device="cuda").to(BF16)
    x[3], x[4] = 1.0, 0.0     # rows as usual beside them; all zeros with eps = 0 is 0/0
    out = binding.add_rmsnorm(x, w, None, eps=0.0, fp8=True, inv_rms=True)
    for r in range(4):
        _check_forward({k: v[r:r + 1] for k, v in out.items()}, x[r:r + 1], None, w, 0.0)
    assert bool(out["y"][4].isnan().all()) and bool(out["y8"][4].float().isnan().all())
    w[:] = 1.0                # infinite products beside finite blocks
    x[0, 3], w[3] = 2.0 ** 100, 2.0 ** 100
    out = binding.add_rmsnorm(x[:1], w, None, eps=0.0, fp8=True)
    assert bool(out["y8"][0, 128:].float().isfinite().all())
