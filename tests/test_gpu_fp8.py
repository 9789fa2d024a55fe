"""Block-scaled e4m3 products (dense and grouped by expert) and the expert layer
in 8 bits, on the GPU against their 64-bit definitions."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from mixture_experts_routed_non_b200 import binding

pytestmark = pytest.mark.gpu

BF16, F32, E8 = torch.bfloat16, torch.float32, torch.float8_e8m0fnu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _linear_case(M, K, N, sa, sw, bias, seed):
    g = _gen(seed)
    a, s = ref.make_rows(g, M, K, sa, "cuda")
    w, t = ref.make_weight(g, 1, N, K, sw, "cuda")
    b = torch.randn((N,), generator=g, device="cuda").to(BF16) if bias else None
    return a, s, w[0], t[0], b


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 100, 127, 128, 129, 256, 300])
@pytest.mark.parametrize("K,N", [(256, 256), (2000, 136)])
def test_linear_rows(M, K, N):
    a, s, w, t, b = _linear_case(M, K, N, E8, E8, M % 2, M)
    y, tol = ref.product(ref.values(a, s), ref.weight_values(w, t), b)
    ref.check(binding.linear_fp8(a, s, w, t, b), y, tol)


@pytest.mark.parametrize("K,N", [(16, 8), (128, 128), (144, 72), (48, 1000), (7168, 264), (1024, 2056), (272, 4096)])
@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("sa,sw", [(E8, E8), (F32, F32), (E8, F32), (F32, E8)])
def test_linear_widths_and_scale_types(K, N, M, sa, sw):
    a, s, w, t, b = _linear_case(M, K, N, sa, sw, True, K + N)
    y, tol = ref.product(ref.values(a, s), ref.weight_values(w, t), b)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref.check(binding.linear_fp8(a, s, w, t, b, err=err), y, tol)
    assert int(err) == 0


# 256-row tiles: rows of scales that are whole words, half-words and odd bytes; partial tiles
@pytest.mark.parametrize("M,K,N", [(1500, 512, 4096), (4097, 384, 2056), (2048, 2048, 2048), (3001, 1376, 1096),
                                   (2500, 768, 2904), (5000, 16, 1288)])
@pytest.mark.parametrize("sc", [E8, F32])
def test_linear_large(M, K, N, sc):
    a, s, w, t, b = _linear_case(M, K, N, sc, sc, True, M)
    y, tol = ref.product(ref.values(a, s), ref.weight_values(w, t), b)
    ref.check(binding.linear_fp8(a, s, w, t, b), y, tol)


# K shared out over clusters of 2, 4 and 8, in even and uneven parts
@pytest.mark.parametrize("K,N", [(1376, 136), (2064, 4096), (4000, 264), (7168, 1024), (11264, 72)])
@pytest.mark.parametrize("M", [1, 9, 32, 61])
@pytest.mark.parametrize("sc", [E8, F32])
def test_linear_split(K, N, M, sc):
    a, s, w, t, b = _linear_case(M, K, N, sc, sc, M == 9, K + M)
    y, tol = ref.product(ref.values(a, s), ref.weight_values(w, t), b)
    out = binding.linear_fp8(a, s, w, t, b)
    ref.check(out, y, tol)
    assert torch.equal(out, binding.linear_fp8(a, s, w, t, b))  # the parts are added in a fixed order


@pytest.mark.parametrize("M", [3, 2000])
def test_linear_scales_at_any_address(M):
    a, s, w, t, _ = _linear_case(M, 1024, 1032, E8, E8, False, 50)
    want = binding.linear_fp8(a, s, w, t)
    for shift in (1, 2, 3):
        def moved(v):
            buf = torch.empty(v.numel() + 8, dtype=torch.uint8, device="cuda")
            buf[shift:shift + v.numel()] = v.view(torch.uint8).flatten()
            return buf[shift:shift + v.numel()].view(E8).view(v.shape)
        assert torch.equal(binding.linear_fp8(a, moved(s), w, moved(t)), want), shift


@pytest.mark.parametrize("M", [1, 40, 700])
def test_linear_nan_codes_and_scales_stay_in_their_rows(M):
    a, s, w, t, _ = _linear_case(M, 384, 256, F32, F32, False, 3)
    clean = binding.linear_fp8(a, s, w, t)
    a.view(torch.uint8)[0, 200] = 0x7F                 # a NaN code
    if M > 30:
        s[29, 1] = float("inf")
        s[30, 2] = float("nan")
    out = binding.linear_fp8(a, s, w, t)
    assert bool(out[0].isnan().all())
    keep = torch.ones(M, dtype=torch.bool)
    keep[0] = False
    if M > 30:
        keep[29:31] = False
        assert not bool(out[29].isfinite().any()) and bool(out[30].isnan().all())
    assert torch.equal(out[keep], clean[keep])


def test_linear_scales_of_any_size():
    """e8m0's end points: 2^-127 and 2^127 as fp32, NaN for 255."""
    a, s, w, t, _ = _linear_case(4, 128, 128, E8, E8, False, 5)
    sb = s.view(torch.uint8)
    sb[:, 0] = torch.tensor([0, 1, 254, 255], dtype=torch.uint8, device="cuda")
    tb = t.view(torch.uint8)
    tb.fill_(127)
    out = binding.linear_fp8(a, s, w, t)
    y = a.float().double() @ w.float().double().T
    mag = a.float().double().abs() @ w.float().double().abs().T
    sc = torch.tensor([2.0 ** -127, 2.0 ** -126, 2.0 ** 127], dtype=torch.float64, device="cuda")[:, None]
    want = (y[:3] * sc)
    over = want.abs() > 3.3e38
    got = out[:3].double()
    assert bool((got.abs()[over] > 3.3e38).all())
    tol = (2.0 ** -8 * y[:3].abs() + ref.product_noise(1) * mag[:3]) * sc + 2.0 ** -133
    ok = (got - want).abs() <= tol
    assert bool((ok | over).all())
    assert bool(out[3].isnan().all())


def test_linear_no_rows():
    a, s, w, t, _ = _linear_case(3, 128, 128, E8, E8, False, 6)
    assert binding.linear_fp8(a[:0], s[:0], w, t).shape == (0, 128)


# --------------------------------------------------------------------------- grouped

SEGMENTS = {
    "one": [1],
    "single_rows": [1, 1, 1, 1],
    "empty_ends": [0, 5, 0, 0, 33, 1, 0],
    "tile_edges": [127, 128, 129, 255, 256, 257, 0, 16, 15, 17],
    "all_in_one": [0, 0, 700, 0],
    "many_small": [i % 5 for i in range(300)],
    "none": [0, 0, 0],
    "long": [2100, 3, 1030],
    "mid": [10, 64, 65, 0, 33, 20, 63, 1],
}


def _grouped_case(counts, K, N, gather, sa, sw, bias, seed, spare=0):
    g = _gen(seed)
    E, used = len(counts), sum(counts)
    P = used + spare
    rows = max(1, P // 3) if gather else P
    a, s = ref.make_rows(g, rows, K, sa, "cuda")
    w, t = ref.make_weight(g, E, N, K, sw, "cuda")
    idx = torch.randint(0, rows, (P,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    b = torch.randn((E, N), generator=g, device="cuda").to(BF16) if bias else None
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    return a, s, off, w, t, b, idx, P


def _grouped_ref(counts, a, s, w, t, b, idx):
    av = ref.values(a, s)
    av = av if idx is None else av[idx.long()]
    y, tol, lo = [], [], 0
    for e, n in enumerate(counts):
        r = ref.product(av[lo:lo + n], ref.weight_values(w[e], t[e]), None if b is None else b[e])
        y.append(r[0]), tol.append(r[1])
        lo += n
    return torch.cat(y), torch.cat(tol)


@pytest.mark.parametrize("name", [n for n in SEGMENTS if n != "none"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K,N", [(256, 256), (208, 136)])
def test_grouped(name, gather, K, N):
    counts = SEGMENTS[name]
    sa, sw = (E8, E8) if N == 256 else (F32, F32)
    a, s, off, w, t, b, idx, P = _grouped_case(counts, K, N, gather, sa, sw, N == 136, len(name), spare=9)
    out = torch.full((P, N), 77.0, dtype=BF16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.grouped_linear_fp8(a, s, off, w, t, b, gather=idx, out=out, err=err)
    assert got is out and int(err) == 0
    y, tol = _grouped_ref(counts, a, s, w, t, b, idx)
    used = sum(counts)
    ref.check(out[:used], y, tol, name)
    assert bool((out[used:] == 77).all())  # rows behind the last segment keep what they held


def test_grouped_empty_segments_write_nothing():
    a, s, off, w, t, b, idx, P = _grouped_case(SEGMENTS["none"], 128, 128, False, E8, E8, False, 1, spare=5)
    out = torch.full((P, 128), 3.0, dtype=BF16, device="cuda")
    binding.grouped_linear_fp8(a, s, off, w, t, out=out)
    assert bool((out == 3).all())


def test_grouped_gather_repeats_and_rows_outside():
    counts = [40, 0, 200]
    a, s, off, w, t, b, idx, P = _grouped_case(counts, 384, 256, True, E8, E8, True, 2)
    idx[:8] = 3
    idx[[20, 100, 230]] = torch.tensor([-1, a.shape[0], 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = binding.grouped_linear_fp8(a, s, off, w, t, b, gather=idx)
    safe = idx.clone()
    safe[[20, 100, 230]] = 0
    y, tol = _grouped_ref(counts, a, s, w, t, b, safe)
    for p in (20, 100, 230):  # counts as zeros: the bias alone
        y[p] = b[0 if p < 40 else 2].double()
        tol[p] = 0
    ref.check(out, y, tol)


def test_grouped_offsets_outside_are_held_inside():
    a, s, off, w, t, b, idx, P = _grouped_case([50, 60], 256, 128, False, E8, E8, False, 3)
    want = binding.grouped_linear_fp8(a, s, off, w, t)
    wild = off.clone()
    wild[0], wild[2] = -5, 10 ** 9
    assert torch.equal(binding.grouped_linear_fp8(a, s, wild, w, t), want)
    down = torch.tensor([50, 50, 0], dtype=torch.int32, device="cuda")  # descending: an empty segment
    out = torch.full_like(want, 5.0)
    binding.grouped_linear_fp8(a, s, down, w, t, out=out)
    assert bool((out == 5).all())


@pytest.mark.parametrize("rows", [60, 700])
def test_grouped_rows_before_the_first_segment_and_overlapping_segments(rows):
    counts = [rows, rows // 2]
    a, s, off, w, t, b, idx, P = _grouped_case(counts, 256, 128, False, E8, E8, False, 6)
    want = binding.grouped_linear_fp8(a, s, off, w, t)
    late = off.clone()
    late[0] = 9  # the first nine rows belong to nobody
    out = torch.full_like(want, 5.0)
    binding.grouped_linear_fp8(a, s, late, w, t, out=out)
    assert bool((out[:9] == 5).all()) and torch.equal(out[9:], want[9:])
    # two experts of the same weight claim every row, with an empty segment between: no row is
    # lost, and none is written outside
    twice = torch.tensor([0, P, 0, P - 3], dtype=torch.int32, device="cuda")
    three = [torch.cat([v.view(torch.uint8), v[:1].view(torch.uint8)]).view(v.dtype) for v in (w, t)]
    out = torch.full_like(want, 5.0)
    binding.grouped_linear_fp8(a, s, twice, *three, out=out)
    y, tol = ref.product(ref.values(a, s), ref.weight_values(w[0], t[0]), None)
    ref.check(out, y, tol)


def test_grouped_many_experts():
    rng = np.random.default_rng(0)
    counts = rng.integers(0, 4, 1024).tolist()
    a, s, off, w, t, b, idx, P = _grouped_case(counts, 128, 128, False, E8, E8, False, 4)
    y, tol = _grouped_ref(counts, a, s, w, t, b, idx)
    ref.check(binding.grouped_linear_fp8(a, s, off, w, t), y, tol)


# --------------------------------------------------------------------------- the layer

def _layer_case(N, H, I, E, K, p_invalid, bias, sx, sw, seed, skew=False):
    g = _gen(seed)
    x, xs = ref.make_rows(g, N, H, sx, "cuda")
    w1, s1 = ref.make_weight(g, E, 2 * I, H, sw, "cuda")
    w2, s2 = ref.make_weight(g, E, H, I, sw, "cuda")
    logits = torch.randn((N, E), generator=g, device="cuda")
    if skew:
        logits += 3 * torch.randn((E,), generator=g, device="cuda")
    idx = logits.topk(K, -1).indices.to(torch.int32).contiguous()
    idx[torch.rand((N, K), generator=g, device="cuda") < p_invalid] = -1
    tw = torch.softmax(torch.randn((N, K), generator=g, device="cuda"), -1)
    tw = torch.where(idx < 0, torch.full_like(tw, float("nan")), tw).contiguous()  # never used
    b1 = torch.randn((E, 2 * I), generator=g, device="cuda").to(BF16) if bias else None
    b2 = torch.randn((E, H), generator=g, device="cuda").to(BF16) if bias else None
    return x, xs, idx, tw, w1, s1, w2, s2, b1, b2


def _layer_ref(x, xs, idx, tw, w1, s1, w2, s2, b1, b2, layout):
    """float64 output and its bound.  h's error (fp32 sums, fast exp and divide) may move a
    value across a rounding border of e4m3: such a value may be off by the codes around it."""
    N, H = x.shape
    E, I2, _ = w1.shape
    I = I2 // 2
    xv = ref.values(x, xs)
    out = torch.zeros((N, H), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    n1, n2 = ref.product_noise(ref.blocks(H)), ref.product_noise(ref.blocks(I))
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        w = ref.weight_values(w1[e], s1[e])
        z, mag = xv[t] @ w.T, xv[t].abs() @ w.abs().T
        if b1 is not None:
            z, mag = z + b1[e].double(), mag + b1[e].double().abs()
        sl = (slice(0, None, 2), slice(1, None, 2)) if layout == binding.LAYOUT_INTERLEAVED else (slice(0, I), slice(I, None))
        gt, up = z[:, sl[0]], z[:, sl[1]]
        silu = gt / (1 + torch.exp(-gt))
        h = silu * up
        # |silu'| < 1.1; exp, divide and product: a few 2^-22 of h
        dh = 1.1 * up.abs() * n1 * mag[:, sl[0]] + silu.abs() * n1 * mag[:, sl[1]] + 2.0 ** -19 * h.abs()
        bl, bd = ref.to_blocks(h), ref.to_blocks(dh)
        s = ref.pow2_scale(bl.abs().amax(-1))
        lo = ref.pow2_scale((bl.abs() - bd).amax(-1).clamp_min(0))
        hi = ref.pow2_scale((bl.abs() + bd).amax(-1))
        q = ref.round_e4m3(bl / s[..., None]) * s[..., None]
        spread = (ref.round_e4m3(((bl + bd) / s[..., None]).clamp(-448, 448))
                  - ref.round_e4m3(((bl - bd) / s[..., None]).clamp(-448, 448))).abs() * s[..., None]
        # where the scale itself is in doubt: half a step in either scale
        unsure = (lo != hi)[..., None] * (2 * (2.0 ** -4 * bl.abs() + 2.0 ** -10 * hi[..., None]))
        hq, dq = q.flatten(-2)[:, :I], (spread + unsure).flatten(-2)[:, :I]
        v = ref.weight_values(w2[e], s2[e])
        y, ym = hq @ v.T, hq.abs() @ v.abs().T
        if b2 is not None:
            y, ym = y + b2[e].double(), ym + b2[e].double().abs()
        # y is kept as fp16 scaled per 32 columns: half a step, or 2^-25 of the scale's range below it
        top = y.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
        dy = dq @ v.abs().T + n2 * ym + 2.0 ** -11 * y.abs() + 2.0 ** -24 * top
        wt = tw[t, k].double()[:, None]
        out.index_add_(0, t, wt * y)
        tol.index_add_(0, t, wt.abs() * (dy * (1 + 2.0 ** -10) + 2.0 ** -20 * y.abs()))
    return out, tol * (1 + 2.0 ** -7) + 2.0 ** -8 * out.abs() + 2.0 ** -133


LAYERS = {
    # N, H, I, E, K, p_invalid, bias, skew
    "one_token": (1, 256, 128, 8, 2, 0.0, False, False),
    "few": (33, 384, 256, 16, 4, 0.3, True, False),
    "decode": (64, 512, 384, 64, 8, 0.1, True, True),
    "rows": (700, 256, 256, 4, 2, 0.2, True, False),
    "skewed": (500, 512, 128, 8, 1, 0.0, False, True),
    "tiles": (1100, 768, 640, 3, 3, 0.05, True, False),
    "mid": (200, 384, 256, 16, 2, 0.1, True, True),
}


@pytest.mark.parametrize("name", LAYERS)
@pytest.mark.parametrize("layout", [binding.LAYOUT_INTERLEAVED, binding.LAYOUT_CONCATENATED])
@pytest.mark.parametrize("sc", [E8, F32])
def test_layer(name, layout, sc):
    N, H, I, E, K, p, bias, skew = LAYERS[name]
    c = _layer_case(N, H, I, E, K, p, bias, sc, sc, 10 + layout, skew)
    y, tol = _layer_ref(*c, layout)
    out = binding.forward_fp8(*c, layout=layout)
    ref.check(out, y, tol, name)


def test_layer_routing_forms_agree():
    N, H, I, E, K = 50, 256, 256, 8, 4
    x, xs, idx, tw, *w = _layer_case(N, H, I, E, K, 0.3, True, E8, E8, 20)
    want = binding.forward_fp8(x, xs, idx, tw, *w)
    P = int((idx >= 0).sum())
    meta = binding.alloc_meta(N, K, E, P)
    assert torch.equal(binding.forward_fp8(x, xs, idx, tw, *w, total_pairs=P, meta=meta), want)
    ref_meta = binding.metadata(idx, tw, E, total_pairs=P)
    for k in ("expert_frequency_offset", "x_gather_idx", "s_reverse_scatter_idx"):
        assert torch.equal(meta[k], ref_meta[k]), k
    assert torch.equal(binding.forward_fp8(x, xs, idx.long(), tw, *w), want)
    t, k = (idx >= 0).nonzero(as_tuple=True)
    got = binding.forward_fp8(x, xs, idx[t, k].contiguous(), tw[t, k].contiguous(), *w, token_idx=t.to(torch.int32))
    assert torch.equal(got, want)


def test_layer_without_pairs_and_without_rows():
    x, xs, idx, tw, *w = _layer_case(9, 256, 128, 4, 2, 0.0, True, E8, E8, 21)
    idx.fill_(-1)
    out = torch.full((9, 256), 4.0, dtype=BF16, device="cuda")
    assert bool((binding.forward_fp8(x, xs, idx, tw, *w, out=out) == 0).all())
    assert binding.forward_fp8(x[:0], xs[:0], idx[:0], tw[:0], *w).shape == (0, 256)


def test_layer_errors_reach_the_workspace():
    N, H, I, E, K = 20, 256, 128, 4, 2
    x, xs, idx, tw, *w = _layer_case(N, H, I, E, K, 0.0, False, E8, E8, 22)
    r = binding.routing(idx, tw)
    ws = torch.empty(binding.fp8_workspace_bytes(r, H, I, E), dtype=torch.uint8, device="cuda")
    want = binding.forward_fp8(x, xs, idx, tw, *w, ws=ws)
    assert binding.read_error(ws) == 0
    bad = idx.clone()
    bad[3, 1] = E
    binding.forward_fp8(x, xs, bad, tw, *w, ws=ws)
    assert binding.read_error(ws) == binding.DEVERR_BAD_EXPERT_ID
    # more pairs than the caller says: nothing is computed, out keeps what it held
    out = torch.full((N, H), 6.0, dtype=BF16, device="cuda")
    binding.forward_fp8(x, xs, idx, tw, *w, total_pairs=N * K - 3, out=out, ws=ws)
    assert binding.read_error(ws) & binding.DEVERR_ABORTED and bool((out == 6).all())
    assert torch.equal(binding.forward_fp8(x, xs, idx, tw, *w, ws=ws), want)


def _block(x, res, nw, rw, idx_w, w1, s1, w2, s2, ws1, ss1, K):
    """One step of a served layer: residual + norm to 8 bits, router, routed experts, a shared
    projection, and the next norm's residual."""
    n = binding.add_rmsnorm(x, nw, res, y=True, fp8=True)
    logits = (n["y"].float() @ rw).contiguous()
    idx, tw = binding.router_topk(logits, K, binding.ROUTER_SOFTMAX_TOPK)
    y = binding.forward_fp8(n["y8"], n["y8_scale"], idx, tw, w1, s1, w2, s2)
    sh = binding.linear_fp8(n["y8"], n["y8_scale"], ws1, ss1)
    return binding.add_rmsnorm(y + sh, nw, n["res"], fp8=True)


@pytest.mark.parametrize("N", [1, 24, 600])
def test_run_together_on_a_stream_and_in_a_graph(N):
    H, I, E, K = 512, 256, 16, 4
    g = _gen(30 + N)
    x = torch.randn((N, H), generator=g, device="cuda").to(BF16)
    res = torch.randn((N, H), generator=g, device="cuda").to(BF16)
    nw = torch.ones(H, dtype=BF16, device="cuda")
    rw = torch.randn((H, E), generator=g, device="cuda") / H ** 0.5
    w1, s1 = binding.quantize_weight_fp8((torch.randn((E, H, 2 * I), generator=g, device="cuda") / H ** 0.5).to(BF16))
    w2, s2 = binding.quantize_weight_fp8((torch.randn((E, I, H), generator=g, device="cuda") / I ** 0.5).to(BF16))
    wsh, ssh = binding.quantize_weight_fp8((torch.randn((H, H), generator=g, device="cuda") / H ** 0.5).to(BF16))
    args = (nw, rw, None, w1, s1, w2, s2, wsh, ssh, K)
    want = _block(x, res, *args)
    torch.cuda.synchronize()

    # against the definition, from the routing and codes the chain itself produced
    n = binding.add_rmsnorm(x, nw, res, y=True, fp8=True)
    idx, tw = binding.router_topk((n["y"].float() @ rw).contiguous(), K, binding.ROUTER_SOFTMAX_TOPK)
    y, tol = _layer_ref(n["y8"], n["y8_scale"], idx, tw, w1, s1, w2, s2, None, None, binding.LAYOUT_INTERLEAVED)
    ref.check(binding.forward_fp8(n["y8"], n["y8_scale"], idx, tw, w1, s1, w2, s2), y, tol)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _block(x, res, *args)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k

    graph = torch.cuda.CUDAGraph()
    xs, rs = x.clone(), res.clone()
    with torch.cuda.graph(graph):
        cap = _block(xs, rs, *args)
    for seed in (1, 2):
        x2 = torch.randn((N, H), generator=_gen(seed), device="cuda").to(BF16)
        xs.copy_(x2)
        graph.replay()
        torch.cuda.synchronize()
        eager = _block(x2, res, *args)
        for k in eager:
            assert torch.equal(cap[k].view(torch.uint8), eager[k].view(torch.uint8)), (seed, k)


def test_layer_on_a_given_stream():
    c = _layer_case(70, 512, 256, 8, 4, 0.1, True, E8, E8, 60)
    want = binding.forward_fp8(*c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [binding.forward_fp8(*c, stream=s) for _ in range(5)]  # workspaces come and go on that stream
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_two_products_on_two_streams():
    a, s, w, t, b = _linear_case(300, 512, 1024, E8, E8, True, 40)
    a2, s2, w2, t2, b2 = _linear_case(3, 2048, 512, E8, E8, True, 41)
    want, want2 = binding.linear_fp8(a, s, w, t, b), binding.linear_fp8(a2, s2, w2, t2, b2)
    torch.cuda.synchronize()
    s1, st2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        outs.append((binding.linear_fp8(a, s, w, t, b, stream=s1), binding.linear_fp8(a2, s2, w2, t2, b2, stream=st2)))
    torch.cuda.synchronize()
    for o, o2 in outs:
        assert torch.equal(o, want) and torch.equal(o2, want2)


@pytest.mark.parametrize("M,K,N", [(100, 7168, 4096), (130, 7168, 4096), (255, 7008, 4088)])
@pytest.mark.parametrize("bias", [False, True])
def test_linear_of_a_hundred_or_two_rows_on_a_large_matrix(M, K, N, bias):
    g = _gen(M + N)
    a, s = ref.make_rows(g, M, K, E8, "cuda")
    w, t = ref.make_weight(g, 1, N, K, E8, "cuda")
    b = torch.randn((N,), generator=g, device="cuda").to(BF16) if bias else None
    out = torch.full((M + 3, N), 9.0, dtype=BF16, device="cuda")
    binding.linear_fp8(a, s, w[0], t[0], b, out=out[:M])
    y, tol = ref.product(ref.values(a, s), ref.weight_values(w[0], t[0]), b)
    ref.check(out[:M], y, tol)
    assert bool((out[M:] == 9).all())


@pytest.mark.parametrize("M,K,N", [(512, 7168, 4096), (256, 7168, 3584), (700, 4640, 888), (1371, 5584, 888), (513, 3600, 264)])
@pytest.mark.parametrize("bias,sa,sw", [(False, E8, E8), (True, E8, E8), (True, F32, F32), (False, E8, F32), (False, F32, E8)])
def test_linear_of_few_tiles_and_a_long_k(M, K, N, bias, sa, sw):
    a, s, w, t, b = _linear_case(M, K, N, sa, sw, bias, M + K)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((M + 3, N), 9.0, dtype=BF16, device="cuda")
    first = binding.linear_fp8(a, s, w, t, b, out=out[:M], err=err).clone()
    y, tol = ref.product(ref.values(a, s), ref.weight_values(w, t), b)
    ref.check(first, y, tol)
    assert bool((out[M:] == 9).all()) and int(err) == 0
    for _ in range(3):  # whatever the pairs' timing
        assert torch.equal(first, binding.linear_fp8(a, s, w, t, b))


@pytest.mark.parametrize("M,K,N", [(96, 2048, 1536), (128, 7168, 512), (256, 7168, 512), (33, 1024, 1200)])
@pytest.mark.parametrize("scale", [E8, F32])
def test_linear_split_over_clusters(M, K, N, scale):
    g = _gen(M + K)
    a, s = ref.make_rows(g, M, K, scale, "cuda")
    w, t = ref.make_weight(g, 1, N, K, scale, "cuda")
    y, tol = ref.product(ref.values(a, s), ref.weight_values(w[0], t[0]), None)
    first = binding.linear_fp8(a, s, w[0], t[0])
    ref.check(first, y, tol)
    assert torch.equal(first, binding.linear_fp8(a, s, w[0], t[0]))


def test_calls_back_to_back_equal_calls_one_by_one():
    """Each call may start while the one before it ends: what it reads (the norm's codes, a
    product's rows, weights quantised just before) and the buffers it writes over are those of
    calls before it, over and over, on one stream and in a graph."""
    g = _gen(77)
    M, H, N = 300, 1024, 640
    x = torch.randn((M, H), generator=g, device="cuda").to(BF16)
    nw = torch.rand((H,), generator=g, device="cuda").to(BF16)
    ws = [(torch.randn(s, generator=g, device="cuda") / s[0] ** 0.5).to(BF16) for s in ((H, N), (N, H))]
    buf = dict(res=torch.empty_like(x), y8=torch.empty((M, H), dtype=torch.float8_e4m3fn, device="cuda"),
               y8_scale=torch.empty((M, H // 128), dtype=E8, device="cuda"))
    qw = [binding.quantize_weight_fp8(w) for w in ws]
    h = torch.empty((M, N), dtype=BF16, device="cuda")
    hq, hs = binding.quantize_rows_fp8(h.zero_())
    o = torch.empty((M, H), dtype=BF16, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty((H,), dtype=F32, device="cuda")
    inv = torch.empty((M,), dtype=F32, device="cuda")
    back = torch.empty(binding.add_rmsnorm_backward_workspace_bytes(M, H), dtype=torch.uint8, device="cuda")

    def run(steps, sync):
        done = torch.cuda.synchronize if sync else lambda: None
        cur, few = x, M
        for i in range(steps):
            few = (M, 17, 130)[i % 3]  # the kernels for long and short segments in turn
            r = binding.add_rmsnorm(x, nw, cur, y=False, fp8=True, inv_rms=True, out=dict(buf, inv_rms=inv)); done()
            binding.quantize_weight_fp8(ws[0], *qw[0]); done()
            binding.linear_fp8(r["y8"][:few], r["y8_scale"][:few], *qw[0], out=h[:few]); done()
            binding.quantize_rows_fp8(h, hq, hs); done()
            binding.linear_fp8(hq, hs, *qw[1], out=o); done()
            binding.add_rmsnorm_backward(o, r["res"], nw, inv, grads=dict(dx=dx, dweight=dw), ws=back); done()
            cur = dx
        return [t.clone() for t in (buf["res"], h, o, dx, dw)]

    h.zero_()
    want = run(30, True)
    for _ in range(3):
        h.zero_()
        for a, b in zip(want, run(30, False)):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(3, False)
        graph = torch.cuda.CUDAGraph()
        h.zero_()
        with torch.cuda.graph(graph, stream=s):
            got = run(30, False)
        for t in (h, o, dx):
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,K,N", [(3, 256, 264), (90, 7168, 4096), (300, 128, 264), (2000, 256, 520)])
@pytest.mark.parametrize("scale", [E8, F32])
def test_bias_at_any_even_address(M, K, N, scale):
    a, s, w, t, b = _linear_case(M, K, N, scale, scale, True, M + 1)
    odd = torch.empty(N + 1, dtype=BF16, device="cuda")[1:]
    odd.copy_(b)
    assert odd.data_ptr() % 16 == 2
    assert torch.equal(binding.linear_fp8(a, s, w, t, odd), binding.linear_fp8(a, s, w, t, b))


def test_layer_bias_at_any_even_address():
    for N in (6, 700):
        x, xs, idx, wt, w1, s1, w2, s2, b1, b2 = _layer_case(N, 256, 128, 5, 2, 0.0, True, E8, E8, 5)
        odd = [torch.empty(b.numel() + 1, dtype=BF16, device="cuda")[1:].view(b.shape) for b in (b1, b2)]
        odd[0].copy_(b1), odd[1].copy_(b2)
        assert odd[0].data_ptr() % 16 == 2
        assert torch.equal(binding.forward_fp8(x, xs, idx, wt, w1, s1, w2, s2, *odd),
                           binding.forward_fp8(x, xs, idx, wt, w1, s1, w2, s2, b1, b2))


_FIRST = """
import torch
from mixture_experts_routed_non_b200 import binding
x = torch.ones((300, 2048), device="cuda").to(torch.bfloat16)
w = torch.ones((2048,), device="cuda").to(torch.bfloat16)
m = torch.ones((2048, 520), device="cuda").to(torch.bfloat16)
off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    r = binding.add_rmsnorm(x, w, y=False, fp8=True, inv_rms=True)
    q, s = binding.quantize_weight_fp8(m)
    few = binding.linear_fp8(r["y8"][:7], r["y8_scale"][:7], q, s)
    all = binding.linear_fp8(r["y8"], r["y8_scale"], q, s)
    two = binding.grouped_linear_fp8(r["y8"], r["y8_scale"], off, torch.stack([q.view(torch.uint8)] * 2).view(q.dtype),
                                     torch.stack([s.view(torch.uint8)] * 2).view(s.dtype))
    g = binding.add_rmsnorm_backward(x, x, w, r["inv_rms"])
graph.replay()
torch.cuda.synchronize()
for y in (few, all, two):
    assert bool((y == 2048).all()), y
print("captured")
"""


def test_first_calls_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_capture_with_two_streams_that_join():
    a, s, w, t, b = _linear_case(300, 1024, 512, E8, E8, False, 3)
    a2, s2, w2, t2, _ = _linear_case(300, 512, 264, E8, E8, False, 4)
    nw = torch.ones((512,), dtype=BF16, device="cuda")
    y1 = binding.linear_fp8(a, s, w, t)
    want = binding.add_rmsnorm(y1, nw, y1, fp8=True)
    want_z = binding.linear_fp8(want["y8"], want["y8_scale"], w2, t2)
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    out = [torch.zeros_like(y1), torch.zeros_like(y1)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        binding.linear_fp8(a, s, w, t, out=out[0])
        with torch.cuda.stream(side):
            binding.linear_fp8(a, s, w, t, out=out[1])
        main.wait_stream(side)
        r = binding.add_rmsnorm(out[0], nw, out[1], fp8=True)  # depends on kernels of both streams
        z = binding.linear_fp8(r["y8"], r["y8_scale"], w2, t2)
    for _ in range(20):
        for o in out:
            o.zero_()
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, want_z) and torch.equal(r["res"], want["res"])


@pytest.mark.parametrize("rows,E,K,N", [(8, 128, 128, 9600), (26700, 3, 128, 4096)])
@pytest.mark.parametrize("scale", [E8, F32])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_more_tiles_than_a_block_lists(rows, E, K, N, scale, gather):
    counts = [rows + (e % 3) - 1 for e in range(E)]  # over 64 units (tiles) to a block (pair)
    a, s, off, w, t, b, idx, P = _grouped_case(counts, K, N, gather, scale, scale, False, 12, spare=2)
    out = torch.full((P, N), 7.0, dtype=BF16, device="cuda")
    binding.grouped_linear_fp8(a, s, off, w, t, gather=idx, out=out)
    assert bool((out[P - 2:] == 7).all())
    ends = off.tolist()
    for e in sorted({0, 1, E // 2, E - 1}):
        p = torch.unique(torch.cat([torch.arange(ends[e], min(ends[e] + 40, ends[e + 1])),
                                    torch.arange(max(ends[e + 1] - 40, ends[e]), ends[e + 1])])).cuda()
        src = p if idx is None else idx[p].long()
        av = ref.values(a.view(torch.uint8)[src].view(a.dtype), s.view(torch.uint8)[src].view(s.dtype)
                        if s.dtype == E8 else s[src])
        y, tol = ref.product(av, ref.weight_values(w[e], t[e]), None)
        ref.check(out[p], y, tol, f"expert {e}")


@pytest.mark.parametrize("counts", [[5, 9], [40, 33], [700, 300]])
@pytest.mark.parametrize("K", [384, 400])
@pytest.mark.parametrize("scale", [E8, F32])
def test_rows_outside_are_zeros_whatever_the_first_and_last_row_hold(counts, K, scale):
    a, s, off, w, t, b, idx, P = _grouped_case(counts, K, 264, True, scale, scale, True, 21)
    rows = a.shape[0]
    idx[(idx == 0) | (idx == rows - 1)] = 1
    want = binding.grouped_linear_fp8(a, s, off, w, t, b, gather=idx)
    for r in (0, rows - 1):  # the rows that stand in for one outside
        a.view(torch.uint8)[r] = 0x7F
        if scale == E8:
            s.view(torch.uint8)[r] = 255
        else:
            s[r] = float("nan")
    bad = torch.arange(0, P, 3, device="cuda")
    idx[bad] = torch.tensor([-1, rows, 2 ** 31 - 1, -(2 ** 31)], dtype=torch.int32, device="cuda").repeat(P)[:len(bad)]
    got = binding.grouped_linear_fp8(a, s, off, w, t, b, gather=idx)
    expert = torch.searchsorted(off[1:].contiguous(), torch.arange(P, device="cuda", dtype=torch.int32), right=True)
    want[bad] = b[expert[bad]]
    assert torch.equal(got, want)
