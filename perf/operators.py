"""Cases that measure the 8-bit path around the expert layer: RMS norm with the
residual's addition (and its gradient), matrix products in 8-bit floating point
with a scale for each block of 128, the same grouped by expert, and the whole
expert layer in 8 bits.

8-bit tensors are e4m3.  A row is scaled per 128 consecutive values, a weight
[N,K] per 128 x 128 block.  Scales are powers of two held as e8m0, or any fp32.
The 8-bit results of the norm come back as the pair (codes as e4m3 values,
scales as e8m0 values), as the framework hands them on.
"""
import math

import torch

own = False

BLOCK = 128
E4M3, E8M0, BF16 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16


def listed():
    return [
        # one decoding token in front of the layer: pure latency
        dict(name="norm_token", op="norm", N=1, H=2048, residual=True, out="fp8"),
        # the prefill workload's rows on their way into the 8-bit layer
        dict(name="norm_prefill_fp8", op="norm", N=16384, H=2048, residual=True, out="fp8"),
        # training rows of the wide layer, an odd number of them: bf16 out, 1/rms kept
        dict(name="norm_train_wide", op="norm", N=8191, H=7168, residual=True, out="train"),
        # gradient of a short odd batch, a width that ends inside a block
        dict(name="norm_back_odd", op="norm_back", N=301, H=1000, dres=False),
        # gradient of the prefill workload's rows, with the residual stream's own gradient
        dict(name="norm_back_prefill", op="norm_back", N=16384, H=2048, dres=True),
        # a shared expert's projection for one decoding token: bound by its weight
        dict(name="linear_token", op="linear", M=1, K=7168, N=4096, bias=False, scale="e8m0"),
        # odd sizes, none a multiple of the block, fp32 scales as a checkpoint may have
        dict(name="linear_odd", op="linear", M=1001, K=2000, N=1496, bias=True, scale="fp32"),
        # a shared expert's projection for the rank-local workload's rows
        dict(name="linear_prefill", op="linear", M=8192, K=7168, N=4096, bias=False, scale="e8m0"),
        # down projection of a decode batch: 256 experts, skewed, many of them empty
        dict(name="grouped_decode", op="grouped", P=1024, E=256, K=512, N=2048, zipf=1.2, gather=False, bias=False, scale="e8m0"),
        # up projection of the prefill workload, rows gathered from the token matrix
        dict(name="grouped_prefill", op="grouped", P=131072, E=128, K=2048, N=1536, zipf=0.0, gather=True, bias=False,
             scale="e8m0"),
        # the whole layer for the decode workload
        dict(name="layer_decode", op="layer", T=128, H=2048, I=512, E=256, topk=8, zipf=1.2, p_invalid=0.0, bias=False),
        # the whole layer for the prefill workload
        dict(name="layer_prefill", op="layer", T=16384, H=2048, I=768, E=128, topk=8, zipf=0.0, p_invalid=0.0, bias=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_back", "linear", "linear", "grouped", "grouped", "layer"])
    if op == "norm":
        H = _log(rng, 64, 7168, 8)
        return dict(op=op, N=_log(rng, 1, 16384 * 2048 // H), H=H, residual=rng.random() < 0.7,
                    out=rng.choice(["fp8", "bf16", "both", "train"]))
    if op == "norm_back":
        H = _log(rng, 64, 7168, 8)
        return dict(op=op, N=_log(rng, 1, 16384 * 2048 // H), H=H, dres=rng.random() < 0.7)
    if op == "linear":
        K, N = _log(rng, 128, 7168, 16), _log(rng, 64, 4096, 8)
        return dict(op=op, M=_log(rng, 1, 8192), K=K, N=N, bias=rng.random() < 0.3, scale=rng.choice(["e8m0", "fp32"]))
    if op == "grouped":
        K, N = _log(rng, 128, 2048, 16), _log(rng, 64, 1536, 8)
        return dict(op=op, P=_log(rng, 1, 65536), E=_log(rng, 1, 256), K=K, N=N, zipf=rng.choice([0.0, 0.8, 1.2]),
                    gather=rng.random() < 0.5, bias=rng.random() < 0.3, scale=rng.choice(["e8m0", "fp32"]))
    E = _log(rng, 8, 256)
    return dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 256, 2048, 128), I=_log(rng, 128, 768, 128), E=E,
                topk=rng.randint(1, 8), zipf=rng.choice([0.0, 1.2]), p_invalid=rng.choice([0.0, 0.3]),
                bias=rng.random() < 0.3)


# --------------------------------------------------------------------------- inputs

def _pad_blocks(v):
    """[..., K] -> [..., ceil(K/128), 128], zeros behind the end."""
    k = v.shape[-1]
    v = torch.nn.functional.pad(v, (0, -k % BLOCK))
    return v.reshape(*v.shape[:-1], -1, BLOCK)


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s; 1 where amax is 0."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))
    return torch.where(amax > 0, s, torch.ones_like(s))


def _quantize(v):
    """fp32 [..., K] -> (e4m3 [..., K], fp32 powers of two [..., ceil(K/128)])."""
    b = _pad_blocks(v)
    s = _pow2_scale(b.abs().amax(-1))
    q = (b / s[..., None]).reshape(*v.shape[:-1], -1)[..., :v.shape[-1]]
    return q.to(E4M3).contiguous(), s


def _make_rows(g, rows, k, scale):
    # activations behind a norm: unit size, a few channels much larger, rows of different loudness
    v = torch.randn((rows, k), generator=g, device="cuda")
    v *= 1 + 15 * (torch.rand((1, k), generator=g, device="cuda") < 0.01)
    v *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    if scale == "fp32":
        s = _pad_blocks(v).abs().amax(-1).clamp_min(1e-6) / 448
        q = _pad_blocks(v) / s[..., None]
        return q.reshape(rows, -1)[:, :k].clamp(-448, 448).to(E4M3).contiguous(), s
    q, s = _quantize(v)
    return q, s.to(E8M0)


def _make_weight(g, e, n, k, scale):
    q = torch.empty((e, n, k), dtype=E4M3, device="cuda")
    s = torch.empty((e, -(-n // BLOCK), -(-k // BLOCK)), device="cuda")
    for i in range(e):
        w = torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k)
        p = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK))
        p = p.reshape(p.shape[0] // BLOCK, BLOCK, p.shape[1] // BLOCK, BLOCK)
        amax = p.abs().amax((1, 3))
        s[i] = amax.clamp_min(1e-12) / 448 if scale == "fp32" else _pow2_scale(amax)
        p = (p / s[i][:, None, :, None]).clamp(-448, 448).to(E4M3)
        q[i] = p.view(torch.uint8).reshape(p.shape[0] * BLOCK, -1)[:n, :k].view(E4M3)
    return q, s if scale == "fp32" else s.to(E8M0)


def _popularity(g, e, zipf):
    rank = torch.randperm(e, generator=g, device="cuda").double() + 1
    return rank.pow(-zipf)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    st = {"case": c}
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    if c["op"] == "norm":
        st["x"] = rand(c["N"], c["H"]).to(BF16)
        st["residual"] = (4 * rand(c["N"], c["H"])).to(BF16) if c["residual"] else None
        st["weight"] = (1 + 0.1 * rand(c["H"])).to(BF16)
    elif c["op"] == "norm_back":
        st["res"] = (4 * rand(c["N"], c["H"])).to(BF16)
        st["weight"] = (1 + 0.1 * rand(c["H"])).to(BF16)
        st["dy"] = rand(c["N"], c["H"]).to(BF16)
        st["dres"] = rand(c["N"], c["H"]).to(BF16) if c["dres"] else None
        st["inv_rms"] = torch.rsqrt(st["res"].double().square().mean(-1) + 1e-6).float()
    elif c["op"] == "linear":
        st["a"], st["a_scale"] = _make_rows(g, c["M"], c["K"], c["scale"])
        w, s = _make_weight(g, 1, c["N"], c["K"], c["scale"])
        st["w"], st["w_scale"] = w[0], s[0]
        st["bias"] = rand(c["N"]).to(BF16) if c["bias"] else None
    elif c["op"] == "grouped":
        share = _popularity(g, c["E"], c["zipf"])
        e = torch.multinomial(share, c["P"], replacement=True, generator=g)
        counts = torch.bincount(e, minlength=c["E"])
        st["counts"] = counts.tolist()  # a dispatch knows them on the host, too
        st["expert_off"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        rows = max(1, c["P"] // 8) if c["gather"] else c["P"]
        st["gather"] = (torch.randint(0, rows, (c["P"],), generator=g, device="cuda", dtype=torch.int32)
                        if c["gather"] else None)
        st["a"], st["a_scale"] = _make_rows(g, rows, c["K"], c["scale"])
        st["w"], st["w_scale"] = _make_weight(g, c["E"], c["N"], c["K"], c["scale"])
        st["bias"] = rand(c["E"], c["N"]).to(BF16) if c["bias"] else None
    else:
        T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["topk"]
        share = _popularity(g, E, c["zipf"])
        gumbel = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda", dtype=torch.float64)))
        idx = torch.topk(gumbel + share.log(), K, dim=-1).indices.to(torch.int32)
        idx[torch.rand((T, K), generator=g, device="cuda") < c["p_invalid"]] = -1
        st["topk_idx"] = idx.contiguous()
        st["topk_w"] = torch.softmax(rand(T, K), -1).contiguous()
        st["counts"] = torch.bincount((idx.reshape(-1) + 1).long(), minlength=E + 1)[1:].tolist()
        st["x"], st["x_scale"] = _make_rows(g, T, H, "e8m0")
        st["w1"], st["w1_scale"] = _make_weight(g, E, 2 * I, H, "e8m0")
        st["w2"], st["w2_scale"] = _make_weight(g, E, H, I, "e8m0")
        st["b1"] = (0.01 * rand(E, 2 * I)).to(BF16) if c["bias"] else None
        st["b2"] = (0.01 * rand(E, H)).to(BF16) if c["bias"] else None
    return st


# --------------------------------------------------------------------------- plain forms

def _rows32(q, s):
    return (q.float().mul_(s.float().repeat_interleave(BLOCK, -1)[..., :q.shape[-1]])
            if q.shape[-1] % BLOCK else
            (q.float().reshape(*s.shape, BLOCK).mul_(s.float()[..., None])).reshape(q.shape))


def _weight32(q, s):
    n, k = q.shape
    return q.float().mul_(s.float().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k])


def _plain_norm(st):
    c, x = st["case"], st["x"]
    out = {}
    if st["residual"] is not None:
        x = (x.float() + st["residual"].float()).to(BF16)
        out["res"] = x
    f = x.float()
    inv = torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)
    y = f * inv * st["weight"].float()
    if c["out"] in ("bf16", "both", "train"):
        out["y"] = y.to(BF16)
    if c["out"] in ("fp8", "both"):
        q, s = _quantize(y)
        out["y8"], out["y8_scale"] = q, s.to(E8M0)
    if c["out"] == "train":
        out["inv_rms"] = inv[:, 0]
    return out


def _plain_norm_back(st):
    s, dy, inv = st["res"].float(), st["dy"].float(), st["inv_rms"][:, None]
    wdy = dy * st["weight"].float()
    hat = s * inv
    dx = inv * (wdy - hat * (wdy * hat).mean(-1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(BF16), "dweight": (dy * hat).sum(0)}


def _plain_grouped(a, counts, w, w_scale, bias):
    # fp32 [P,N]: one product for each expert that has rows
    return torch.cat([r @ _weight32(w[e], w_scale[e]).T + (0 if bias is None else bias[e].float())
                      for e, r in enumerate(torch.split(a, counts)) if len(r)])


def _plain_layer(st):
    c = st["case"]
    T, H, E, K = c["T"], c["H"], c["E"], c["topk"]
    out = torch.zeros((T * K, H), device="cuda")
    if sum(st["counts"]):
        e = st["topk_idx"].reshape(-1)
        order = torch.argsort(torch.where(e < 0, E, e), stable=True)[:sum(st["counts"])]
        z = _plain_grouped(_rows32(st["x"], st["x_scale"])[order // K], st["counts"], st["w1"], st["w1_scale"], st["b1"])
        gate, up = z[:, 0::2], z[:, 1::2]
        h = gate * torch.sigmoid(gate) * up
        y = _plain_grouped(_rows32(*_quantize(h)), st["counts"], st["w2"], st["w2_scale"], st["b2"])
        out[order] = y * st["topk_w"].reshape(-1)[order, None]
    return out.reshape(T, K, H).sum(1).to(BF16)


def run(st):
    c = st["case"]
    if own:
        from mixture_experts_routed_non_b200 import binding
        if c["op"] == "norm":
            return binding.add_rmsnorm(st["x"], st["weight"], st["residual"], eps=1e-6, y=c["out"] != "fp8",
                                       fp8=c["out"] in ("fp8", "both"), inv_rms=c["out"] == "train")
        if c["op"] == "norm_back":
            return binding.add_rmsnorm_backward(st["dy"], st["res"], st["weight"], st["inv_rms"], dres=st["dres"])
        if c["op"] == "linear":
            return binding.linear_fp8(st["a"], st["a_scale"], st["w"], st["w_scale"], st["bias"])
        if c["op"] == "grouped":
            return binding.grouped_linear_fp8(st["a"], st["a_scale"], st["expert_off"], st["w"], st["w_scale"],
                                              st["bias"], gather=st["gather"])
        return binding.forward_fp8(st["x"], st["x_scale"], st["topk_idx"], st["topk_w"], st["w1"], st["w1_scale"],
                                   st["w2"], st["w2_scale"], st["b1"], st["b2"])
    if c["op"] == "norm":
        return _plain_norm(st)
    if c["op"] == "norm_back":
        return _plain_norm_back(st)
    if c["op"] == "linear":
        y = _rows32(st["a"], st["a_scale"]) @ _weight32(st["w"], st["w_scale"]).T
        return (y if st["bias"] is None else y + st["bias"].float()).to(BF16)
    if c["op"] == "grouped":
        a = _rows32(st["a"], st["a_scale"])
        return _plain_grouped(a if st["gather"] is None else a[st["gather"].long()], st["counts"], st["w"],
                              st["w_scale"], st["bias"]).to(BF16)
    return _plain_layer(st)


# --------------------------------------------------------------------------- definition in 64 bits

def _e4m3_64(v):
    """Nearest e4m3 value, ties to even, of float64 values within +-448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _codes_64(v):
    """float64 [..., K] -> codes and scales by the definition."""
    k = v.shape[-1]
    whole = torch.zeros((*v.shape[:-1], -(-k // BLOCK) * BLOCK), dtype=torch.float64, device=v.device)
    whole[..., :k] = v
    whole = whole.unflatten(-1, (-1, BLOCK))
    amax = whole.abs().max(-1).values
    s = torch.exp2(torch.ceil(torch.log2(amax / 448)))
    s = torch.where(amax <= 448 * s / 2, s / 2, s)  # log2 may be off at an exact power
    s = torch.where(amax > 448 * s, s * 2, s)
    s = torch.where(amax == 0, torch.ones_like(s), s)
    return _e4m3_64(whole / s[..., None]).flatten(-2)[..., :k], s


def _values_64(q, s):
    return q.double() * torch.repeat_interleave(s.double(), BLOCK, dim=-1)[..., :q.shape[-1]]


def _weight_64(q, s):
    i = torch.arange(q.shape[0], device=q.device) // BLOCK
    j = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * s.double()[i][:, j]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        s, out = st["x"], {}
        if st["residual"] is not None:
            s = (s.double() + st["residual"].double()).float().to(BF16)
            out["res"] = s.double()
        d = s.double()
        inv = 1 / torch.sqrt((d * d).sum(-1) / case["H"] + 1e-6)
        y = d * st["weight"].double() * inv[:, None]
        if case["out"] != "fp8":
            out["y"] = y
        if case["out"] in ("fp8", "both"):
            out["y8"], out["y8_scale"] = _codes_64(y)
        if case["out"] == "train":
            out["inv_rms"] = inv
        return out
    if op == "norm_back":
        s, dy, w, inv = st["res"].double(), st["dy"].double(), st["weight"].double(), st["inv_rms"].double()
        c = (dy * w * s).sum(-1) / case["H"]
        dx = dy * w * inv[:, None] - s * (inv ** 3 * c)[:, None]
        if st["dres"] is not None:
            dx += st["dres"].double()
        return {"dx": dx, "dweight": (dy * s * inv[:, None]).sum(0)}
    if op == "linear":
        y = _values_64(st["a"], st["a_scale"]) @ _weight_64(st["w"], st["w_scale"]).T
        return y if st["bias"] is None else y + st["bias"].double()
    if op == "grouped":
        a = _values_64(st["a"], st["a_scale"])
        y = torch.empty((case["P"], case["N"]), dtype=torch.float64, device="cuda")
        lo = 0
        for e, n in enumerate(st["counts"]):
            if n:
                rows = a[lo:lo + n] if st["gather"] is None else a[st["gather"][lo:lo + n].long()]
                y[lo:lo + n] = rows @ _weight_64(st["w"][e], st["w_scale"][e]).T
                if st["bias"] is not None:
                    y[lo:lo + n] += st["bias"][e].double()
            lo += n
        return y
    x = _values_64(st["x"], st["x_scale"])
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    for e, n in enumerate(st["counts"]):
        if not n:
            continue
        t, k = torch.nonzero(st["topk_idx"] == e, as_tuple=True)
        z = x[t] @ _weight_64(st["w1"][e], st["w1_scale"][e]).T
        if st["b1"] is not None:
            z += st["b1"][e].double()
        codes, s = _codes_64(z[:, 0::2] / (1 + torch.exp(-z[:, 0::2])) * z[:, 1::2])
        r = _values_64(codes, s) @ _weight_64(st["w2"][e], st["w2_scale"][e]).T
        if st["b2"] is not None:
            r += st["b2"][e].double()
        y.index_add_(0, t, r * st["topk_w"][t, k, None].double())
    return y


# --------------------------------------------------------------------------- work

def _blocks(n):
    return -(-n // BLOCK)


def _active(P, E, zipf):
    """Experts with rows, expected: by the popularities of the draw."""
    share = [r ** -zipf for r in range(1, E + 1)]
    total = sum(share)
    return sum(1 - (1 - v / total) ** P for v in share)


def work(case):
    c = case
    if c["op"] == "norm":
        N, H = c["N"], c["H"]
        b = 2 * N * H + 2 * H + (4 * N * H if c["residual"] else 0)
        b += 2 * N * H if c["out"] != "fp8" else 0
        b += N * H + N * _blocks(H) if c["out"] in ("fp8", "both") else 0
        return {"bytes": b + (4 * N if c["out"] == "train" else 0), "flops": 5 * N * H}
    if c["op"] == "norm_back":
        N, H = c["N"], c["H"]
        return {"bytes": 2 * N * H * (4 if c["dres"] else 3) + 4 * N + 6 * H, "flops": 10 * N * H}
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        sb = 4 if c["scale"] == "fp32" else 1
        return {"bytes": M * K + N * K + sb * _blocks(K) * (M + _blocks(N)) + 2 * M * N + (2 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    if c["op"] == "grouped":
        P, E, K, N = c["P"], c["E"], c["K"], c["N"]
        rows, act = max(1, P // 8) if c["gather"] else P, _active(P, E, c["zipf"])
        sb = 4 if c["scale"] == "fp32" else 1
        return {"bytes": rows * (K + sb * _blocks(K)) + act * (N * K + sb * _blocks(N) * _blocks(K)) + 2 * P * N
                + (4 * P if c["gather"] else 0) + 4 * (E + 1) + (2 * act * N if c["bias"] else 0),
                "flops": 2 * P * N * K}
    T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["topk"]
    P = T * K * (1 - c["p_invalid"])
    act = _active(P, E, c["zipf"])
    return {"bytes": T * (H + _blocks(H)) + 8 * T * K + act * 3 * H * I + 2 * T * H
            + (act * (4 * I + 2 * H) if c["bias"] else 0), "flops": 6 * P * H * I}
