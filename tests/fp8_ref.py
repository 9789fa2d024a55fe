"""64-bit definitions of the norm, the 8-bit quantisation and the block-scaled
products, and the rounding bounds the parity tests hold the kernels to.

A rounding is off by at most half a step: 2^-8 of the value in bf16, 2^-11 in
fp16, 2^-24 in fp32, 2^-4 in e4m3 (2^-10 of the scale below e4m3's normal
range, whose step is 2^-9)."""
import torch

BLOCK = 128
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def blocks(n):
    return -(-n // BLOCK)


def to_blocks(v):
    """[..., K] -> [..., ceil(K/128), 128], zeros behind the end."""
    k = v.shape[-1]
    p = torch.zeros(v.shape[:-1] + (blocks(k) * BLOCK,), dtype=v.dtype, device=v.device)
    p[..., :k] = v
    return p.unflatten(-1, (-1, BLOCK))


def pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s; 1 at 0; at least 2^-126 (float64)."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875))
    s = torch.where(amax == 0, torch.ones_like(s), s)
    return s.clamp_min(2.0 ** -126)


def round_e4m3(v):
    """float64 -> nearest e4m3 value, ties to even; non-finite -> NaN.  |v| <= 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.where(torch.isfinite(v), torch.round(v / step) * step, torch.full_like(v, float("nan")))


def quantize(v):
    """float64 [..., K] -> (code values [..., K], scales [..., ceil(K/128)])."""
    b = to_blocks(v)
    s = pow2_scale(torch.where(torch.isfinite(b), b.abs(), torch.zeros_like(b)).amax(-1))
    return round_e4m3(b / s[..., None]).flatten(-2)[..., :v.shape[-1]], s


def values(q, s):
    """Codes and their scales -> float64 values, scales repeated along the last axis."""
    s = s.float().double()
    return q.float().double() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def weight_values(q, s):
    n, k = q.shape[-2:]
    s = s.float().double().repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]
    return q.float().double() * s


def make_rows(g, m, k, scale, device):
    v = torch.randn((m, k), generator=g, device=device) * torch.exp(torch.randn((m, 1), generator=g, device=device))
    if scale == torch.float32:
        s = (to_blocks(v).abs().amax(-1) / 448).clamp_min(1e-9)
        q = (to_blocks(v) / s[..., None]).flatten(-2)[:, :k].clamp(-448, 448)
        return q.to(E4M3).contiguous(), s
    q, s = quantize(v.double())
    return q.float().to(E4M3).contiguous(), s.float().to(E8M0)


def make_weight(g, e, n, k, scale, device):
    v = torch.randn((e, n, k), generator=g, device=device) / k ** 0.5
    p = torch.zeros((e, blocks(n) * BLOCK, blocks(k) * BLOCK), device=device)
    p[:, :n, :k] = v
    p = p.view(e, blocks(n), BLOCK, blocks(k), BLOCK)
    amax = p.abs().amax((2, 4))
    s = (amax / 448).clamp_min(1e-12) if scale == torch.float32 else pow2_scale(amax.double()).float()
    q = (p / s[:, :, None, :, None]).clamp(-448, 448).reshape(e, blocks(n) * BLOCK, -1)[:, :n, :k]
    q = q.to(E4M3).contiguous()
    return q, s if scale == torch.float32 else s.to(E8M0)


def product_noise(nk):
    """Relative to sum |a||w|, for nk blocks of 128: products of e4m3 codes are exact in fp32, and
    every addition or scaling is off by no more than a whole fp32 step.  Summed block by block: 128
    additions inside a block, nk of blocks, two scalings.  Summed through (32 values of K per matrix
    instruction, scales applied to the products): 32 additions inside an instruction, 4 nk of
    instructions, at most 8 of the K split's parts.  Both stay below 128 + 4 nk."""
    return (128 + 4 * nk) * 2.0 ** -23


def product(a, w, bias=None):
    """float64 a [M,K] . w [N,K]^T + bias, and the bound of the bf16 result's error."""
    y = a @ w.T
    mag = a.abs() @ w.abs().T
    if bias is not None:
        y = y + bias.double()
        mag = mag + bias.double().abs()
    tol = 2.0 ** -8 * y.abs() + product_noise(blocks(a.shape[1])) * (1 + 2.0 ** -8) * mag + 2.0 ** -133
    return y, tol


def check(got, ref, tol, what=""):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0].item()} for {ref[bad][0].item()} "
                           f"+- {tol[bad][0].item()}")


def norm(x, residual, weight, eps):
    """(s as float64 of the rounded bf16 sum, inv, y)."""
    s = x.double() if residual is None else (x.float() + residual.float()).to(torch.bfloat16).double()
    inv = 1 / torch.sqrt(s.square().mean(-1) + eps)
    return s, inv, s * inv[:, None] * weight.double()


def norm_backward(dy, s, weight, inv, dres=None):
    """float64 (dx, dweight) by the formula."""
    c = (dy * weight * s).mean(-1, keepdim=True)
    dx = inv[:, None] * weight * dy - inv[:, None] ** 3 * c * s
    return dx if dres is None else dx + dres, (dy * s * inv[:, None]).sum(0)
