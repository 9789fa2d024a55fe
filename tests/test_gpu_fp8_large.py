"""The norm, the row quantiser and the 8-bit products where element offsets pass 32 bits: the first and the last
rows against the 64-bit definitions."""
import pytest
import torch

import fp8_ref as ref
from mixture_experts_routed_non_b200 import binding
from test_gpu_norm import FP32, _check_forward

pytestmark = pytest.mark.gpu

BF16, F32, E8, E4 = torch.bfloat16, torch.float32, torch.float8_e8m0fnu, torch.float8_e4m3fn
ROWS, COLS = 530000, 4104   # 2.2e9 values, past 2^31
K = 8320                    # ROWS x K: 4.4e9 bytes of codes, past 2^32
ENDS = [slice(0, 200), slice(ROWS - 200, ROWS)]


@pytest.fixture(autouse=True)
def _room():
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(shape, seed):
    """e4m3 codes of magnitudes up to 1.875, both signs."""
    q = torch.randint(0, 64, shape, generator=_gen(seed), dtype=torch.uint8, device="cuda")
    q |= torch.randint(0, 2, (shape[-1],), generator=_gen(seed + 1), dtype=torch.uint8, device="cuda") << 7
    return q.view(E4)


def _scales(shape, dtype, seed):
    b = torch.randint(120, 134, shape, generator=_gen(seed), dtype=torch.uint8, device="cuda").view(E8)
    return b if dtype == E8 else b.float() * 1.37


def _rows(t, rows):
    return t.view(torch.uint8)[rows].view(t.dtype) if t.dtype in (E4, E8) else t[rows]


@pytest.mark.parametrize("scale", [E8, F32])
def test_linear_and_gathered_rows(scale):
    a, s = _codes((ROWS, K), 1), _scales((ROWS, K // 128), scale, 2)
    w, t = _codes((COLS, K), 3), _scales((ref.blocks(COLS), K // 128), scale, 4)
    out = binding.linear_fp8(a, s, w, t)
    wv = ref.weight_values(w, t)
    for rows in ENDS:
        y, tol = ref.product(ref.values(_rows(a, rows), _rows(s, rows)), wv)
        ref.check(out[rows], y, tol)
    del out
    # few gathered rows: the other kernels' loads of the same rows
    idx = torch.tensor([ROWS - 1, 0, ROWS - 7, 5, ROWS - 2], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    w2 = torch.stack([w[:264].view(torch.uint8)] * 2).view(E4)
    t2 = torch.stack([t[:3].view(torch.uint8) if scale == E8 else t[:3]] * 2)
    t2 = t2.view(E8) if scale == E8 else t2
    out = binding.grouped_linear_fp8(a, s, off, w2, t2, gather=idx)
    y, tol = ref.product(ref.values(_rows(a, idx.long()), _rows(s, idx.long())), wv[:264])
    ref.check(out, y, tol)


def test_norm_quantiser_and_gradient():
    g = _gen(7)
    x = torch.randn((ROWS, COLS), generator=g, device="cuda", dtype=BF16)
    r = torch.randn((ROWS, COLS), generator=g, device="cuda", dtype=BF16)
    w = (1 + 0.3 * torch.randn((COLS,), generator=g, device="cuda")).to(BF16)
    f = binding.add_rmsnorm(x, w, r, y=True, fp8=True, inv_rms=True, eps=1e-5)
    for rows in ENDS:
        _check_forward({k: _rows(v, rows) for k, v in f.items()}, x[rows], r[rows], w, 1e-5)
    del f["y8"], f["y8_scale"]
    b = binding.add_rmsnorm_backward(x, f["res"], w, f["inv_rms"], dres=r, grads=dict(dx=f["y"]))
    for rows in ENDS:
        d, s, inv, dres = x[rows].double(), f["res"][rows].double(), f["inv_rms"][rows].double(), r[rows].double()
        dx, _ = ref.norm_backward(d, s, w.double(), inv, dres)
        mag = ((inv[:, None] * w.double() * d).abs() + dres.abs()
               + inv[:, None] ** 3 * (d * w.double() * s).abs().mean(-1, keepdim=True) * s.abs())
        ref.check(b["dx"][rows], dx, 2.0 ** -8 * dx.abs() + 2 * FP32 * mag + 2.0 ** -133, "dx")
    del b, f, r
    x = x.view(-1)[:ROWS * 4096].view(ROWS, 4096)
    q, sc = binding.quantize_rows_fp8(x)
    for rows in ENDS:
        want, ws = ref.quantize(x[rows].double())
        assert torch.equal(_rows(q, rows).float().double(), want) and torch.equal(_rows(sc, rows).float().double(), ws)
