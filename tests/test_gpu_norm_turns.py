"""The norm and its gradient where each block takes several turns at its ring of row loads: stages loaded
again while rows are worked on, in place too, against the 64-bit definitions."""
import pytest
import torch

import fp8_ref as ref
from mixture_experts_routed_non_b200 import binding
from test_gpu_norm import FP32, _check_forward, _gen, _inputs

pytestmark = pytest.mark.gpu

# N, H: at least three turns for each of the (at most 1184) blocks, the last ones of few rows; one, two and four
# chunks of columns per thread, rows that share a block and rows that do not, a width that ends inside a block
TURNS = [(30001, 128), (30007, 136), (15001, 2048), (7999, 1032), (3701, 7168), (2001, 8200), (1801, 16384)]


@pytest.mark.parametrize("N,H", TURNS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kw", [dict(fp8=True, inv_rms=True), dict(y=False, fp8=True)])
def test_forward(N, H, residual, kw):
    x, r, w = _inputs(N, H, N + H)
    out = binding.add_rmsnorm(x, w, r if residual else None, eps=1e-5, **kw)
    _check_forward(out, x, r if residual else None, w, 1e-5)


@pytest.mark.parametrize("N,H", TURNS)
def test_forward_in_place(N, H):
    x, r, w = _inputs(N, H, N + 1)
    want = binding.add_rmsnorm(x, w, r, inv_rms=True)
    x2, r2 = x.clone(), r.clone()
    got = binding.add_rmsnorm(x2, w, r2, inv_rms=True, out=dict(res=r2, y=x2))  # rows are loaded ahead of what is written
    _check_forward(got, x, r, w, 1e-6)
    assert all(torch.equal(got[k], want[k]) for k in want)


# at least three turns for each of 296 blocks
@pytest.mark.parametrize("N,H", [(15001, 128), (8003, 136), (2001, 2048), (1999, 1032), (1001, 7168), (901, 8200), (899, 16384)])
@pytest.mark.parametrize("with_dres", [False, True])
def test_backward(N, H, with_dres):
    x, r, w = _inputs(N, H, N)
    g = _gen(H)
    dy = torch.randn((N, H), generator=g, device="cuda").to(torch.bfloat16)
    dres = torch.randn((N, H), generator=g, device="cuda").to(torch.bfloat16) if with_dres else None
    f = binding.add_rmsnorm(x, w, r, inv_rms=True)
    over = dy.clone()
    got = binding.add_rmsnorm_backward(over, f["res"], w, f["inv_rms"], dres=dres, grads=dict(dx=over))  # in place
    s, inv = f["res"].double(), f["inv_rms"].double()
    d, wd = dy.double(), w.double()
    dx, dw = ref.norm_backward(d, s, wd, inv, None if dres is None else dres.double())
    mag = (inv[:, None] * wd * d).abs() + inv[:, None] ** 3 * (d * wd * s).abs().mean(-1, keepdim=True) * s.abs()
    if dres is not None:
        mag = mag + dres.double().abs()
    ref.check(got["dx"], dx, 2.0 ** -8 * dx.abs() + 2 * FP32 * mag + 2.0 ** -133, "dx")
    # a row's term: two roundings (the product with inv, the sum); a block's turns one after the other: at most
    # N / 296 + 1 where a row has the block for itself; 15 sums of its row groups; 296 blocks in 32 sums of
    # at most 10, then 5 levels of a tree
    steps = 1 + (N // 296 + 1) + 15 + 10 + 5
    ref.check(got["dweight"], dw, steps * 2.0 ** -24 * 1.01 * (d * s * inv[:, None]).abs().sum(0) + 2.0 ** -140, "dweight")


def test_backward_of_rows_whose_1_over_rms_squared_passes_the_range():
    """1 / rms = 2^65: its square is no fp32 number, the gradient is."""
    N, H = 5, 640
    g = _gen(3)
    sign = torch.where(torch.rand((N, H), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x = (sign * 2.0 ** -65).to(torch.bfloat16)
    x[3] = 1.0  # a row as usual beside them
    w = (1 + 0.3 * torch.randn((H,), generator=g, device="cuda")).to(torch.bfloat16)
    dy = torch.randn((N, H), generator=g, device="cuda").to(torch.bfloat16)
    inv = binding.add_rmsnorm(x, w, eps=0.0, inv_rms=True)["inv_rms"]
    assert bool((inv[:3] == 2.0 ** 65).all())
    got = binding.add_rmsnorm_backward(dy, x, w, inv)
    s, d, wd, i = x.double(), dy.double(), w.double(), inv.double()
    dx, dw = ref.norm_backward(d, s, wd, i)
    mag = (i[:, None] * wd * d).abs() + i[:, None] ** 3 * (d * wd * s).abs().mean(-1, keepdim=True) * s.abs()
    ref.check(got["dx"], dx, 2.0 ** -8 * dx.abs() + 2 * FP32 * mag, "dx")
    ref.check(got["dweight"], dw, 2.0 ** -18 * (d * s * i[:, None]).abs().sum(0), "dweight")
