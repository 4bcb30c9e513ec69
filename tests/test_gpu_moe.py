"""The router, the slots' order by expert and the rows' way to the experts and back
against plain implementations in 64 bits: experts, counts, orders and moved rows
exactly, weights and sums within bounds derived from their roundings."""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from layer_util import f64, generator, host_bits, normal, outs

pytestmark = pytest.mark.gpu

U8, F32, BF16, I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32
HALF = 2.0 ** -24


# ---- the router ------------------------------------------------------------------

def scores64(l, sigmoid):
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            e = np.exp(-np.abs(l))
            return np.where(l >= 0, 1 / (1 + e), e / (1 + e))
        m = l.max(1, keepdims=True)
        e = np.where(m == -np.inf, 0.0, np.exp(l - np.where(m == -np.inf, 0.0, m)))
        s = e.sum(1, keepdims=True)
        return e / np.where(s > 0, s, 1.0)


def route64(l, bias, top, flags, groups, top_groups, scale):
    """experts and weights, token by token, from the definition."""
    T, E = l.shape
    p = scores64(l, flags & mx.ROUTE_SIGMOID)
    pair = bool(flags & mx.ROUTE_GROUP_PAIR) and groups > 1
    key = l.copy() if bias is None and not pair else p + (0.0 if bias is None else bias)
    key[(l == -np.inf) | (np.zeros(E) if bias is None else bias == -np.inf).astype(bool)] = -np.inf
    ex, w = np.full((T, top), -1), np.zeros((T, top))
    S = E // groups
    for t in range(T):
        k = key[t].copy()
        if groups > 1:
            best = []
            for g in range(groups):
                v = np.sort(k[g * S:(g + 1) * S])[::-1]
                best.append(v[0] + (v[1] if pair and S > 1 and v[1] > -np.inf else 0.0))
            order = sorted(range(groups), key=lambda g: (-best[g], g))
            for g in order[top_groups:]:
                k[g * S:(g + 1) * S] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-k[e], e)) if k[e] > -np.inf][:top]
        ex[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
    if flags & mx.ROUTE_RENORM:
        s = w.sum(1, keepdims=True)
        w = w / np.where(s > 0, s, 1.0)
    return ex, w * scale, p


def check_route(logits, top, bias=None, flags=0, groups=1, top_groups=1, scale=1.0):
    T, E = logits.shape
    buf, broken = outs(dict(experts=((T, top), I32), weights=((T, top), F32), scores=((T, E), F32)))
    o = mx.moe_route(logits.cuda(), top, bias=None if bias is None else bias.cuda(), flags=flags,
                     groups=groups, top_groups=top_groups, scale=scale, want_scores=True, out=buf)
    torch.cuda.synchronize()
    assert broken() == []
    sc = float(np.float32(scale))
    ex, w, p = route64(f64(logits), None if bias is None else f64(bias), top, flags, groups, top_groups, sc)
    assert np.array_equal(o["experts"].cpu().numpy(), ex)
    # exp: 2 ulp; a softmax sum of E terms in at most E / 64 + 6 additions; division,
    # the product with the reciprocal; the sum of the chosen ones (7), division, scale
    adds = -(-E // 64) + 6
    tol = (2 * 4 + adds + 4) * HALF
    # (below fp32's normal numbers, 2^-149 at a time)
    assert np.all(np.abs(f64(o["scores"]) - p) <= tol * p + 2.0 ** -148)
    tol = (2 * tol / HALF + 7 + 2) * HALF
    assert np.all(np.abs(f64(o["weights"]) - w) <= tol * np.abs(w) + 2.0 ** -148 * max(1, abs(sc)))
    return o


def logits_of(g, T, E, dtype=F32, masked=0.0, scale=2.0):
    x = torch.randn(T, E, generator=g) * scale
    if masked:
        x[torch.rand(T, E, generator=g) < masked] = float("-inf")
    return x.to(dtype)


ROUTES = [(1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (5, 4, 4, 2, 1), (33, 64, 6, 8, 3), (17, 40, 5, 4, 2),
          (9, 128, 8, 8, 4), (6, 160, 6, 8, 3), (7, 256, 8, 8, 4), (64, 256, 1, 1, 1), (3, 500, 10, 5, 2),
          (5, 512, 8, 16, 4), (3, 1024, 64, 32, 8), (4, 1000, 33, 1, 1), (130, 63, 7, 1, 1),
          (2, 64, 64, 64, 9), (3, 65, 65 - 1, 1, 1), (3, 1023, 9, 3, 1), (2, 96, 8, 48, 20), (2, 1024, 64, 64, 64)]


@pytest.mark.parametrize("T,E,top,groups,kept", ROUTES)
@pytest.mark.parametrize("sigmoid", [0, mx.ROUTE_SIGMOID], ids=["softmax", "sigmoid"])
def test_route(T, E, top, groups, kept, sigmoid):
    g = generator(T * 31 + E)
    bias = torch.randn(E, generator=g) * 0.1
    for dtype in (F32, BF16):
        l = logits_of(g, T, E, dtype)
        check_route(l, top, flags=sigmoid, scale=1.0)
        check_route(l, top, flags=sigmoid | mx.ROUTE_RENORM, groups=groups, top_groups=kept, scale=2.5)
        check_route(l, top, bias, flags=sigmoid | mx.ROUTE_RENORM, groups=groups, top_groups=kept)
        check_route(l, top, bias, flags=sigmoid | mx.ROUTE_GROUP_PAIR, groups=groups, top_groups=kept,
                    scale=-0.5)
        check_route(l, top, flags=sigmoid | mx.ROUTE_GROUP_PAIR | mx.ROUTE_RENORM, groups=groups,
                    top_groups=kept)


@pytest.mark.parametrize("E,groups", [(16, 4), (64, 8), (256, 8), (600, 6)])
@pytest.mark.parametrize("flags", [0, mx.ROUTE_SIGMOID, mx.ROUTE_RENORM | mx.ROUTE_GROUP_PAIR,
                                   mx.ROUTE_SIGMOID | mx.ROUTE_RENORM | mx.ROUTE_GROUP_PAIR])
def test_route_with_masked_experts(E, groups, flags):
    """Rows with few experts or none, whole groups masked, experts masked by bias."""
    g = generator(E)
    l = logits_of(g, 40, E, masked=0.9)
    l[3] = float("-inf")
    l[4] = float("-inf")
    l[4, E - 1] = -3.0
    l[5, : E // groups] = float("-inf")
    l[6] = -3.4e38
    l[7, 0] = -3.4e38
    bias = torch.randn(E, generator=g) * 0.2
    bias[:: 5] = float("-inf")
    for b in (None, bias):
        o = check_route(l, min(8, E), b, flags=flags, groups=groups, top_groups=2)
        assert bool((o["experts"][3] == -1).all()) and bool((o["weights"][3] == 0).all())


@pytest.mark.parametrize("flags", [0, mx.ROUTE_SIGMOID])
def test_route_ties_go_to_the_lowest_index(flags):
    l = torch.zeros(6, 256)
    l[1, 100:] = 1.0
    l[2] = torch.arange(256) // 2 % 3
    l[3, 0::2] = -0.0
    l[4] = 50.0
    o = check_route(l, 10, flags=flags)
    assert o["experts"][0].tolist() == list(range(10))
    assert o["experts"][1].tolist() == list(range(100, 110))
    for pair in (0, mx.ROUTE_GROUP_PAIR):
        o = check_route(l, 6, torch.zeros(256), flags=flags | pair, groups=8, top_groups=2)
        assert o["experts"][0].tolist() == list(range(6))


def test_route_keys_next_to_each_other():
    """Biases that part keys by 2^-40 of them decide, those that make them equal in
    64 bits do not: fp32 scores would not tell any of these apart."""
    E = 64
    l = torch.full((1, E), 0.25)
    bias = torch.full((E,), 2.0 ** -60)
    bias[40] = 2.0 ** -40
    bias[7] = 2.0 ** -41
    for sig in (0, mx.ROUTE_SIGMOID):
        o = check_route(l, 3, bias, flags=sig)
        assert o["experts"][0].tolist() == [40, 7, 0]


@pytest.mark.parametrize("E", [8, 256])
@pytest.mark.parametrize("flags", [mx.ROUTE_RENORM, mx.ROUTE_SIGMOID | mx.ROUTE_RENORM])
def test_route_nan_stays_in_its_row(E, flags):
    g = generator(2)
    l = logits_of(g, 9, E)
    want = mx.moe_route(l.cuda(), 4, flags=flags)
    l[2, E - 1] = float("nan")
    l[5] = float("nan")
    o = mx.moe_route(l.cuda(), 4, flags=flags, groups=2, top_groups=2, want_scores=True)
    torch.cuda.synchronize()
    for t in range(9):
        if t in (2, 5):
            assert bool((o["experts"][t] == -1).all()) and bool(o["weights"][t].isnan().all())
        else:
            assert torch.equal(o["experts"][t], want["experts"][t])
            assert torch.equal(o["weights"][t], want["weights"][t])
    inf = logits_of(g, 3, E)
    inf[1, 3] = float("inf")
    o = mx.moe_route(inf.cuda(), 2, flags=flags)
    if flags & mx.ROUTE_SIGMOID:
        assert o["experts"][1, 0].item() == 3 and bool(o["weights"].isfinite().all())
    else:
        assert bool((o["experts"][1] == -1).all()) and bool(o["weights"][1].isnan().all())


@pytest.mark.parametrize("E,groups", [(32, 4), (256, 8), (300, 5)])
def test_route_of_nan_in_masked_places(E, groups):
    """A NaN bias of an expert whose logit is -Inf, a NaN logit of one whose bias is
    (by sigmoid scores, which stand alone): neither is seen."""
    g = generator(E)
    l = logits_of(g, 20, E)
    bias = torch.randn(E, generator=g) * 0.1
    l[:, 3] = float("-inf")
    bias[3] = float("nan")
    bias[7] = float("-inf")
    l2, b2 = l.clone(), bias.clone()
    b2[3] = 0.0
    for flags in (0, mx.ROUTE_SIGMOID, mx.ROUTE_SIGMOID | mx.ROUTE_GROUP_PAIR | mx.ROUTE_RENORM):
        if flags & mx.ROUTE_SIGMOID:
            l[:, 7] = float("nan")
        a = mx.moe_route(l.cuda(), 5, bias=bias.cuda(), flags=flags, groups=groups, top_groups=2)
        b = mx.moe_route(l2.cuda(), 5, bias=b2.cuda(), flags=flags, groups=groups, top_groups=2)
        assert bool((a["experts"] >= 0).all())
        assert torch.equal(a["experts"], b["experts"]) and torch.equal(a["weights"], b["weights"])


def test_route_with_an_infinite_bias():
    """+Inf: those experts first, the lowest index first among them; -Inf: never."""
    g = generator(3)
    for E in (16, 256, 300):
        l = logits_of(g, 6, E)
        bias = torch.zeros(E)
        bias[9] = bias[5] = float("inf")
        bias[2] = float("-inf")
        for flags in (0, mx.ROUTE_SIGMOID):
            o = mx.moe_route(l.cuda(), 4, bias=bias.cuda(), flags=flags)
            assert bool((o["experts"][:, 0] == 5).all()) and bool((o["experts"][:, 1] == 9).all())
            assert not bool((o["experts"] == 2).any()) and bool(o["weights"].isfinite().all())


def test_route_with_large_biases():
    """Keys of every magnitude: the fixed point's steps grow with the largest bias."""
    g = generator(8)
    for scale in (1e-6, 30.0, 1e6, 1e30, 3e38):
        l, bias = logits_of(g, 50, 64), torch.randn(64, generator=g) * min(scale, 1e37)
        bias[0] = scale
        check_route(l, 6, bias, flags=mx.ROUTE_SIGMOID)
        check_route(l, 6, bias, groups=8, top_groups=3, flags=mx.ROUTE_GROUP_PAIR if scale < 1e37 else 0)


def grad64(l, ex, dw, ds, flags, scale):
    p = scores64(l, flags & mx.ROUTE_SIGMOID)
    T, E = l.shape
    dp = np.zeros((T, E)) if ds is None else ds.copy()
    chosen = np.zeros((T, E))
    for t in range(T):
        js = [j for j in range(ex.shape[1]) if 0 <= ex[t, j] < E]
        es = [ex[t, j] for j in js]
        d = scale * dw[t, js]
        if flags & mx.ROUTE_RENORM:
            s = p[t, es].sum()
            d = (d - (d * p[t, es]).sum() / s) / s if s > 0 else 0 * d
        for e, v in zip(es, d):
            dp[t, e] += v
            chosen[t, e] += abs(v)
    if flags & mx.ROUTE_SIGMOID:
        return dp * p * scores64(-l, True), p, chosen
    return p * (dp - (dp * p).sum(1, keepdims=True)), p, chosen


def check_route_back(l, ex, flags, scale, ds=False, seed=0):
    T, E = l.shape
    g = generator(seed)
    dw = torch.randn(ex.shape, generator=g)
    ds = torch.randn(T, E, generator=g) if ds else None
    buf, broken = outs(dict(out=((T, E), l.dtype)))
    o = mx.moe_route_backward(dw.cuda(), l.cuda(), ex.cuda(), flags=flags, scale=scale,
                              dscores=None if ds is None else ds.cuda(), out=buf["out"])
    torch.cuda.synchronize()
    assert broken() == []
    sc = float(np.float32(scale))
    want, p, chosen = grad64(f64(l), ex.numpy(), f64(dw), None if ds is None else f64(ds), flags, sc)
    # p carries tol, the chosen ones' gradients (sums over the chosen of d p / s: up to
    # three p, 20 roundings) their magnitude before they cancel
    tol = (8 + -(-E // 64) + 10) * HALF
    mag = np.zeros((T, E))
    for t in range(T):
        es = [e for e in ex[t].tolist() if 0 <= e < E]
        s = p[t, es].sum() if flags & mx.ROUTE_RENORM else 1.0
        top = abs(sc) * np.abs(f64(dw)[t]).max() if len(es) else 0.0
        mag[t, es] = 2 * top / s * len(es) if s > 0 else 0.0
    mag += 0 if ds is None else np.abs(f64(ds))
    if flags & mx.ROUTE_SIGMOID:
        bound = p * scores64(-f64(l), True) * mag
    else:
        bound = p * (mag + (p * mag).sum(1, keepdims=True))
    half = 2.0 ** -8 if l.dtype == BF16 else HALF
    bound = half * np.abs(want) + (4 * tol + 24 * HALF) * bound + 1e-37
    assert np.all(np.abs(f64(o) - want) <= bound)
    return f64(o)


@pytest.mark.parametrize("T,E,top,groups,kept", ROUTES)
@pytest.mark.parametrize("flags", [0, 1, 2, 3])
def test_route_backward(T, E, top, groups, kept, flags):
    g = generator(E * 3 + T)
    for dtype in (F32, BF16):
        l = logits_of(g, T, E, dtype, masked=0.2)
        ex = mx.moe_route(l.cuda(), top, flags=flags)["experts"].cpu()
        check_route_back(l, ex, flags, 1.0, seed=1)
        d = check_route_back(l, ex, flags, -1.5, ds=True, seed=2)
        assert np.all(d[f64(l) == -np.inf] == 0)


def test_route_backward_of_other_experts():
    """Indices outside the experts, and the same one twice (it counts twice)."""
    g = generator(4)
    l = logits_of(g, 4, 16)
    ex = torch.tensor([[3, 3, 5], [-1, 16, 2], [-1, -1, -1], [2 ** 31 - 1, -2 ** 31, 0]], dtype=I32)
    for flags in range(4):
        d = check_route_back(l, ex, flags, 1.0, seed=flags)
        assert np.all(d[2] == 0)


@pytest.mark.parametrize("E", [16, 256, 600])
@pytest.mark.parametrize("flags", [0, 1, 2, 3])
def test_route_backward_ignores_masked_places(E, flags):
    g = generator(E + flags)
    l = logits_of(g, 10, E, masked=0.4)
    ex = mx.moe_route(l.cuda(), 4, flags=flags)["experts"]
    dw, ds = torch.randn(10, 4, generator=g).cuda(), torch.randn(10, E, generator=g)
    clean = mx.moe_route_backward(dw, l.cuda(), ex, flags=flags, dscores=ds.cuda())
    ds[l == float("-inf")] = float("nan")
    o = mx.moe_route_backward(dw, l.cuda(), ex, flags=flags, dscores=ds.cuda())
    assert torch.equal(o, clean) and bool((o[l.cuda() == float("-inf")] == 0).all())


@pytest.mark.parametrize("flags", [0, 1, 2, 3])
def test_route_backward_against_differences(flags):
    """Against central differences of sum(dw w) + sum(ds p) in 64 bits with the choice
    held fixed (step 1e-4: off by less than 1e-7 of the gradients)."""
    g = generator(6)
    T, E, top, step = 2, 12, 3, 1e-4
    l = logits_of(g, T, E)
    ex = mx.moe_route(l.cuda(), top, flags=flags)["experts"].cpu()
    dw, ds = torch.randn(T, top, generator=g), torch.randn(T, E, generator=g)
    got = f64(mx.moe_route_backward(dw.cuda(), l.cuda(), ex.cuda(), flags=flags, scale=2.0,
                                    dscores=ds.cuda()))

    def loss(x):
        p = scores64(x, flags & 1)
        w = np.take_along_axis(p, ex.numpy().astype(np.int64), 1)
        if flags & 2:
            w = w / w.sum(1, keepdims=True)
        return (2.0 * w * f64(dw)).sum() + (p * f64(ds)).sum()

    for t in range(T):
        for e in range(E):
            d = np.zeros((T, E))
            d[t, e] = step
            num = (loss(f64(l) + d) - loss(f64(l) - d)) / (2 * step)
            assert abs(got[t, e] - num) <= 1e-5


# ---- the order of the slots ---------------------------------------------------------

def sort_ref(ex, E, align, rows):
    flat = ex.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(E)])
    pos, slots, at = np.full(flat.shape, -1), np.full(rows, -1), 0
    for e in np.nonzero(counts)[0]:
        start = int((-(-counts[:e] // align) * align).sum())
        idx = np.nonzero(flat == e)[0]
        pos[idx] = start + np.arange(len(idx))
        slots[start:start + len(idx)] = idx
    return counts, pos.reshape(ex.shape), slots


def experts_of(seed, T, top, E, none=0.0, skew=False):
    r = np.random.default_rng(seed)
    ex = (r.random((T, top)) ** 3 * E).astype(np.int32) if skew else r.integers(0, E, (T, top), dtype=np.int32)
    if none:
        off = r.random((T, top)) < none
        ex[off] = r.choice([-1, E, 2 ** 31 - 1, -2 ** 31], off.sum())
    return torch.from_numpy(ex)


def check_sort(ex, E, align, more=0):
    T, top = ex.shape
    rows = mx.moe_sort_rows(T, top, E, align) + more
    buf, broken = outs(dict(counts=((E,), I32), pos=((T, top), I32), slots=((rows,), I32)))
    o = mx.moe_sort(ex.cuda(), E, align=align, rows=rows, out=buf)
    torch.cuda.synchronize()
    assert broken() == []
    for k, want in zip(("counts", "pos", "slots"), sort_ref(ex.numpy(), E, align, rows)):
        assert np.array_equal(o[k].cpu().numpy(), want), k
    return o


@pytest.mark.parametrize("T,top,E", [(1, 1, 1), (1, 8, 8), (3, 2, 5), (64, 1, 64), (65, 1, 2), (128, 4, 16),
                                     (1000, 8, 256), (1024, 8, 1024), (1025, 8, 7), (4096, 4, 8), (4097, 4, 9),
                                     (128, 8, 256), (129, 8, 1024), (512, 8, 31), (513, 8, 64), (2048, 8, 1000),
                                     (2049, 8, 5), (4096, 8, 128), (4097, 8, 1000), (8193, 8, 300), (65536, 1, 3),
                                     (5000, 3, 1000), (20001, 8, 64), (70000, 7, 33), (8193, 1, 1)])
def test_sort(T, top, E):
    check_sort(experts_of(T, T, top, E), E, 1)
    check_sort(experts_of(T + 1, T, top, E, none=0.3, skew=True), E, 16, more=77)
    check_sort(torch.full((T, top), E - 1, dtype=I32), E, 32)
    check_sort(torch.full((T, top), -1, dtype=I32), E, 128, more=1)


def test_sort_of_many_slots():
    """2^23 slots: every workgroup takes 64 times 512."""
    ex = experts_of(9, 1 << 17, 64, 256)
    o = mx.moe_sort(ex.cuda(), 256, align=16)
    torch.cuda.synchronize()
    flat = ex.reshape(-1).long()
    counts = torch.bincount(flat, minlength=256)
    assert torch.equal(o["counts"].cpu().long(), counts)
    order = torch.argsort(flat, stable=True)
    padded = (counts + 15) // 16 * 16
    start, first = padded.cumsum(0) - padded, counts.cumsum(0) - counts
    e = flat[order]
    row = start[e] + torch.arange(flat.numel()) - first[e]
    pos = torch.empty_like(flat)
    pos[order] = row
    assert torch.equal(o["pos"].cpu().view(-1).long(), pos)
    slots = torch.full((o["slots"].numel(),), -1)
    slots[row] = order
    assert torch.equal(o["slots"].cpu().long(), slots)


# ---- rows -----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,width", [(BF16, 1), (BF16, 8), (BF16, 7), (BF16, 4096), (BF16, 1111),
                                         (U8, 1), (U8, 33), (U8, 7168), (F32, 130), (torch.float64, 1025),
                                         (U8, 70000)])
def test_gather(dtype, width):
    for T, top, rows in ((1, 1, 1), (5, 3, 20), (300, 2, 700)):
        g = generator(width + T)
        x = torch.randint(0, 256, (T, width * torch.empty(0, dtype=dtype).element_size()), generator=g,
                          dtype=torch.int32).to(U8).view(dtype)
        slots = torch.randint(-2, T * top + 2, (rows,), generator=g, dtype=I32)
        slots[0] = T * top - 1
        buf, broken = outs(dict(out=((rows, width), dtype)))
        o = mx.moe_gather(x.cuda(), slots.cuda(), top, out=buf["out"])
        torch.cuda.synchronize()
        assert broken() == []
        live = (slots >= 0) & (slots < T * top)
        want = torch.zeros(rows, width, dtype=dtype)
        want[live] = x[(slots[live] // top).long()]
        assert torch.equal(o.cpu().view(U8), want.view(U8))


@pytest.mark.parametrize("T,top,rows", [(9000, 2, 140000), (9000, 4, 140000), (8100, 2, 20001)])
def test_gather_of_many_rows(T, top, rows):
    """Both orders of the rows, more of them than the grid has workgroups."""
    g = torch.Generator("cuda").manual_seed(rows + top)
    x = torch.randint(0, 256, (T, 8192), generator=g, device="cuda", dtype=torch.int32).to(U8)
    slots = torch.randint(-2, T * top + 2, (rows,), generator=g, device="cuda", dtype=I32)
    o = mx.moe_gather(x, slots, top)
    live = (slots >= 0) & (slots < T * top)
    at = (slots // top).clamp(0, T - 1).long()
    for r in range(0, rows, 10000):
        want = torch.where(live[r:r + 10000, None], x[at[r:r + 10000]], x.new_zeros(()))
        assert torch.equal(o[r:r + 10000], want)


def rows_case(T, top, E, align, K, seed, none=0.1):
    g = generator(seed)
    ex = experts_of(seed, T, top, E, none=none)
    s = mx.moe_sort(ex.cuda(), E, align=align)
    R = s["slots"].numel()
    return dict(y=normal(g, R, K), w=torch.randn(T, top, generator=g), pos=s["pos"], slots=s["slots"],
                dout=normal(g, T, K))


def combine_ref(y, w, pos):
    T, top = pos.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for j in range(top):
        live = (pos[:, j] >= 0) & (pos[:, j] < len(y))
        v = w[live, j:j + 1] * y[pos[live, j]]
        out[live] += v
        mag[live] += np.abs(v)
    return out, mag


COMBINE = [(1, 1, 1, 1, 8), (1, 8, 8, 1, 4096), (5, 2, 4, 16, 1), (33, 4, 8, 16, 2056), (64, 3, 7, 1, 1111),
           (200, 8, 64, 32, 512), (7, 64, 100, 1, 24), (300, 1, 5, 8, 7168)]


@pytest.mark.parametrize("T,top,E,align,K", COMBINE)
def test_combine(T, top, E, align, K):
    c = rows_case(T, top, E, align, K, T + K)
    # a fused product and addition per slot, half a step of bf16
    for w in (c["w"], None):
        buf, broken = outs(dict(out=((T, K), BF16)))
        o = mx.moe_combine(c["y"].cuda(), None if w is None else w.cuda(), c["pos"], out=buf["out"])
        torch.cuda.synchronize()
        assert broken() == []
        want, mag = combine_ref(f64(c["y"]), np.ones((T, top)) if w is None else f64(w),
                                c["pos"].cpu().numpy())
        assert np.all(np.abs(f64(o) - want) <= 2.0 ** -8 * np.abs(want) + top * HALF * mag * 1.01 + 1e-38)
    y3 = normal(generator(K), T, top, K)
    o = mx.moe_combine(y3.cuda(), c["w"].cuda())
    want = (f64(y3) * f64(c["w"])[:, :, None]).sum(1)
    mag = np.abs(f64(y3) * f64(c["w"])[:, :, None]).sum(1)
    assert np.all(np.abs(f64(o) - want) <= 2.0 ** -8 * np.abs(want) + top * HALF * mag * 1.01 + 1e-38)


def test_combine_at_every_end_of_a_row():
    for K in (*range(1, 18), *range(2041, 2058)):
        g = generator(K)
        y, w, dout = normal(g, 7, K), torch.randn(5, 2, generator=g), normal(g, 5, K)
        pos = torch.tensor([[0, 6], [-1, 2], [3, 3], [7, 1], [5, 4]], dtype=I32)
        slots = torch.tensor([0, 7, 3, 4, 9, 8, 1], dtype=I32)
        bufs, broken = outs(dict(out=((5, K), BF16), dy=((7, K), BF16), dweights=((5, 2), F32)))
        o = mx.moe_combine(y.cuda(), w.cuda(), pos.cuda(), out=bufs["out"])
        b = mx.moe_combine_backward(dout.cuda(), y.cuda(), w.cuda(), pos=pos.cuda(), slots=slots.cuda(),
                                    out=bufs)
        torch.cuda.synchronize()
        assert broken() == []
        want, mag = combine_ref(f64(y), f64(w), pos.numpy())
        assert np.all(np.abs(f64(o) - want) <= 2.0 ** -8 * np.abs(want) + 2 * HALF * mag * 1.01 + 1e-38)
        s = slots.numpy()
        dy = f64(w).reshape(-1)[s, None] * f64(dout)[s // 2]
        assert np.all(np.abs(f64(b["dy"]) - dy) <= (2.0 ** -8 + 2 * HALF) * np.abs(dy))
        p = pos.numpy()
        live = (p >= 0) & (p < 7)
        prod = np.where(live[:, :, None], f64(y)[np.where(live, p, 0)], 0.0) * f64(dout)[:, None, :]
        adds = 8 * -(-K // 512) + 7
        assert np.all(np.abs(f64(b["dweights"]) - prod.sum(2)) <= adds * HALF * np.abs(prod).sum(2) + 1e-38)


def test_combine_of_any_positions():
    """Rows named twice or by no slot, positions outside the rows."""
    g = generator(12)
    y, w = normal(g, 6, 40), torch.randn(4, 3, generator=g)
    pos = torch.tensor([[0, 0, 5], [6, -1, 3], [2 ** 31 - 1, -2 ** 31, -7], [5, 4, 4]], dtype=I32)
    o = mx.moe_combine(y.cuda(), w.cuda(), pos.cuda())
    want, mag = combine_ref(f64(y), f64(w), pos.numpy())
    assert np.all(np.abs(f64(o) - want) <= 2.0 ** -8 * np.abs(want) + 4 * HALF * mag)
    assert np.all(f64(o)[2] == 0)


@pytest.mark.parametrize("T,top,E,align,K", COMBINE)
def test_combine_backward(T, top, E, align, K):
    c = rows_case(T, top, E, align, K, T + K + 1)
    R = c["y"].shape[0]
    pos, slots, dout, y = c["pos"].cpu().numpy(), c["slots"].cpu().numpy(), f64(c["dout"]), f64(c["y"])
    for w in (c["w"], None):
        buf, broken = outs(dict(dy=((R, K), BF16), dweights=((T, top), F32)))
        o = mx.moe_combine_backward(c["dout"].cuda(), c["y"].cuda(), None if w is None else w.cuda(),
                                    pos=c["pos"], slots=c["slots"], out=buf)
        torch.cuda.synchronize()
        assert broken() == []
        wt = np.ones((T, top)) if w is None else f64(w)
        live = slots >= 0
        dy = np.zeros((R, K))
        dy[live] = wt.reshape(-1)[slots[live], None] * dout[slots[live] // top]
        assert np.all(np.abs(f64(o["dy"]) - dy) <= (2.0 ** -8 + 2 * HALF) * np.abs(dy))
        assert np.all(f64(o["dy"])[~live] == 0)
        prod = np.where((pos >= 0)[:, :, None], y[np.maximum(pos, 0)], 0.0) * dout[:, None, :]
        adds = 8 * -(-K // 512) + 7         # a lane's products in a line, 8 of every 512; 6 over the wave
        assert np.all(np.abs(f64(o["dweights"]) - prod.sum(2)) <= adds * HALF * np.abs(prod).sum(2) + 1e-38)
    y3 = normal(generator(K), T, top, K)
    o = mx.moe_combine_backward(c["dout"].cuda(), y3.cuda(), c["w"].cuda())
    assert o["dy"].shape == y3.shape
    want = f64(c["w"])[:, :, None] * dout[:, None, :]
    assert np.all(np.abs(f64(o["dy"]) - want) <= (2.0 ** -8 + 2 * HALF) * np.abs(want))


def test_combine_backward_of_other_orders():
    """Rows whose slot does not name them back are left as they were; a row named by
    two slots is its own slot's; a slot without a row has no gradient."""
    g = generator(13)
    y, w, dout = normal(g, 5, 16), torch.randn(2, 3, generator=g), normal(g, 2, 16)
    pos = torch.tensor([[0, 0, 1], [9, -1, 3]], dtype=I32)
    slots = torch.tensor([1, 2, 4, 5, -1], dtype=I32)       # row 2's slot has no row
    dy = torch.full((5, 16), 7.0, dtype=BF16, device="cuda")
    o = mx.moe_combine_backward(dout.cuda(), y.cuda(), w.cuda(), pos=pos.cuda(), slots=slots.cuda(),
                                out=dict(dy=dy))
    wd, d = f64(w), f64(dout)
    for r, want in ((0, wd[0, 1] * d[0]), (1, wd[0, 2] * d[0]), (3, wd[1, 2] * d[1]), (4, 0 * d[0])):
        assert np.all(np.abs(f64(o["dy"])[r] - want) <= 2.0 ** -8 * np.abs(want) * 1.01), r
    assert np.all(f64(o["dy"])[2] == 7)
    dw = f64(o["dweights"])
    yd = f64(y)
    want = np.array([[d[0] @ yd[0], d[0] @ yd[0], d[0] @ yd[1]], [0, 0, d[1] @ yd[3]]])
    assert np.all(np.abs(dw - want) <= 1e-5)


def test_combine_backward_without_dweights():
    c = rows_case(40, 3, 5, 4, 72, 3)
    args = (c["dout"].cuda(), c["y"].cuda(), c["w"].cuda())
    a = mx.moe_combine_backward(*args, pos=c["pos"], slots=c["slots"])
    b = mx.moe_combine_backward(*args, pos=c["pos"], slots=c["slots"], want_dweights=False)
    assert b["dweights"] is None and torch.equal(a["dy"], b["dy"])


def test_codes_and_scales_take_the_same_way():
    """A row-wise cast's codes and compact scales, moved instead of bf16 rows: the cast
    of the moved rows."""
    g = generator(15)
    T, top, K = 70, 2, 200
    x = normal(g, T, K).cuda()
    s = mx.moe_sort(experts_of(5, T, top, 4, none=0.1).cuda(), 4, align=16)
    c = mx.mx_quantize(x, axis=mx.ROWWISE)
    want = mx.mx_quantize(mx.moe_gather(x, s["slots"], top), axis=mx.ROWWISE)
    assert torch.equal(mx.moe_gather(c["q_row"], s["slots"], top), want["q_row"])
    assert torch.equal(mx.moe_gather(c["s_row"], s["slots"], top), want["s_row"])


def test_gather_and_combine_are_each_others_gradient():
    """<combine(y, 1), g> = <y, gather(g)> in 64 bits, on whole numbers (exact)."""
    g = generator(14)
    T, top, K = 50, 4, 136
    s = mx.moe_sort(experts_of(3, T, top, 6, none=0.2).cuda(), 6, align=8)
    y = torch.randint(-3, 4, (s["slots"].numel(), K), generator=g).to(BF16).cuda()
    d = torch.randint(-3, 4, (T, K), generator=g).to(BF16).cuda()
    a = (f64(mx.moe_combine(y, pos=s["pos"])) * f64(d)).sum()
    b = (f64(y) * f64(mx.moe_gather(d, s["slots"], top))).sum()
    assert a == b


def test_rows_past_32_bit_offsets():
    """More than 2^32 bytes of rows: the last ones, there and back."""
    T, top, K, R = 131200, 2, 8200, 262400
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    x[-3:] = torch.arange(3 * K, device="cuda").view(3, K).to(BF16)
    w = torch.ones(T, top, device="cuda")
    w[-3:, 1] = 2.0
    ex = torch.zeros(T, top, dtype=I32, device="cuda")
    ex[:, 1] = 1
    s = mx.moe_sort(ex, 2)
    assert s["slots"].numel() == R and s["pos"][-1].tolist() == [T - 1, R - 1]
    xs = mx.moe_gather(x, s["slots"], top)
    assert torch.equal(xs[T - 3:T], x[-3:]) and torch.equal(xs[-3:], x[-3:])
    assert not bool(xs[T:-3].any()) and not bool(xs[:T - 3].any())
    out = mx.moe_combine(xs, w, s["pos"])
    assert torch.equal(out[-3:], (3 * x[-3:].float()).to(BF16)) and not bool(out[:-3].any())
    b = mx.moe_combine_backward(x, xs, w, pos=s["pos"], slots=s["slots"])
    assert torch.equal(b["dy"][-3:], (2 * x[-3:].float()).to(BF16))
    assert torch.equal(b["dy"][T - 3:T], x[-3:]) and not bool(b["dy"][T:-3].any())
    want = (x[-3:].double() ** 2).sum(1)
    adds = 8 * -(-K // 512) + 7
    assert bool(((b["dweights"][-3:].double() - want[:, None]).abs() <= adds * HALF * want[:, None]).all())


# ---- together, streams, graphs -----------------------------------------------------------

def layer(x, res, wn, wr, bias, wq, N, top, E, stream=None):
    """One decoded batch: norm, router, the experts' 4-bit products, back."""
    n = mx.mx_rmsnorm(x, wn, residual=res, stream=stream)
    y = n["y"]
    logits = (y.float() @ wr.float())
    r = mx.moe_route(logits, top, bias=bias, flags=mx.ROUTE_SIGMOID | mx.ROUTE_RENORM, groups=2,
                     top_groups=1, scale=2.0, stream=stream)
    p = mx.nvfp4_matvec_experts(y, r["experts"], wq["q_row"], wq["s_row"], wq["sg"], stream=stream)
    return dict(out=mx.moe_combine(p, r["weights"], stream=stream), experts=r["experts"], h=n["h"],
                weights=r["weights"], p=p, y=y)


def test_decode_through_the_layer():
    g = generator(20)
    T, K, N, E, top = 6, 256, 96, 8, 3
    x, res, wn = (normal(g, *s).cuda() for s in ((T, K), (T, K), (K,)))
    wr, bias = normal(g, K, E).cuda(), (torch.randn(E, generator=g) * 0.1).cuda()
    w = normal(g, E * N, K).cuda()
    wq = mx.nvfp4_quantize_transpose_grouped(w, [N] * E, mx.mx_absmax_bf16_grouped(w, [N] * E),
                                             axis=mx.ROWWISE)
    o = layer(x, res, wn, wr, bias, wq, N, top, E)
    torch.cuda.synchronize()
    want = (f64(o["p"]) * f64(o["weights"])[:, :, None]).sum(1)
    mag = np.abs(f64(o["p"]) * f64(o["weights"])[:, :, None]).sum(1)
    assert np.all(np.abs(f64(o["out"]) - want) <= 2.0 ** -8 * np.abs(want) + 4 * HALF * mag)
    assert bool((o["experts"] >= 0).all())
    # captured and replayed, with new inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x, res, wn, wr, bias, wq, N, top, E)
    for seed in (21, 22, 23):
        h = generator(seed)
        x.copy_(normal(h, T, K))
        res.copy_(normal(h, T, K))
        graph.replay()
        torch.cuda.synchronize()
        again = layer(x, res, wn, wr, bias, wq, N, top, E)
        torch.cuda.synchronize()
        for k in ("out", "experts", "h", "weights"):
            assert torch.equal(got[k], again[k]), (seed, k)


def test_training_step_through_the_experts():
    """Router, order, rows, grouped cast and product, back, and the gradients down to
    the tokens and the logits, against the same steps in 64 bits on the operands as
    cast (whole chain: the grouped product's own bounds, then half steps of bf16)."""
    g = generator(30)
    T, K, N, E, top, align = 200, 128, 64, 4, 2, 16
    x, w, logits = normal(g, T, K).cuda(), normal(g, E * N, K).cuda(), logits_of(g, T, E).cuda()
    r = mx.moe_route(logits, top, flags=mx.ROUTE_RENORM)
    s = mx.moe_sort(r["experts"], E, align=align)
    rows = [-(-int(c) // align) * align for c in s["counts"].tolist()]
    M = sum(rows)
    slots = s["slots"][:M].contiguous()
    xs = mx.moe_gather(x, slots, top)
    cx, cw = mx.mx_quantize_grouped(xs, rows), mx.mx_quantize_grouped(w, [N] * E)
    y = mx.mx_matmul_grouped(cx["q_row"], cx["s_row"], cw["q_row"], cw["s_row"], rows)
    out = mx.moe_combine(y, r["weights"], s["pos"])
    dout = normal(g, T, N).cuda()
    b = mx.moe_combine_backward(dout, y, r["weights"], pos=s["pos"], slots=slots)
    cd = mx.mx_quantize_grouped(b["dy"], rows)
    dw = mx.mx_matmul_wgrad_grouped(cd["q_col"], cd["s_col"], cx["q_col"], cx["s_col"], rows,
                                    flags=mx.OUT_F32)
    dlogits = mx.moe_route_backward(b["dweights"], logits, r["experts"], flags=mx.ROUTE_RENORM)
    torch.cuda.synchronize()
    # against 64 bits, expert by expert: E4M3 operands are off by 2^-4, half of it in
    # the sum of squares at most, so that sums of 128 products agree to a tenth
    xf, wf, pos = f64(x), f64(w).reshape(E, N, K), s["pos"].cpu().numpy()
    ex, wt = r["experts"].cpu().numpy(), f64(r["weights"])
    ref = np.zeros((T, N))
    for j in range(top):
        ref += wt[:, j:j + 1] * np.einsum("tk,tnk->tn", xf, wf[ex[:, j]])
    assert np.linalg.norm(f64(out) - ref) <= 0.1 * np.linalg.norm(ref)
    # the steps around the product, on what it gave
    yd = f64(y)
    want = sum(wt[:, j:j + 1] * yd[pos[:, j]] for j in range(top))
    mag = sum(np.abs(wt[:, j:j + 1] * yd[pos[:, j]]) for j in range(top))
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + 4 * HALF * mag)
    assert np.all(np.isfinite(f64(dw))) and np.all(np.isfinite(f64(dlogits)))
    # rows of padding: no gradient, nothing in the weight gradients
    live = slots.cpu().numpy() >= 0
    assert not f64(b["dy"])[~live].any() and not f64(xs)[~live].any()
    grad, _, _ = grad64(f64(logits), ex, f64(b["dweights"]), None, mx.ROUTE_RENORM, 1.0)
    assert np.all(np.abs(f64(dlogits) - grad) <= 1e-4 * np.abs(f64(b["dweights"])).max())


def test_sort_and_rows_in_a_graph_and_on_a_stream():
    g = generator(40)
    T, top, E, K = 3000, 4, 32, 264
    ex = experts_of(1, T, top, E, none=0.1).cuda()
    x, wt, dout = normal(g, T, K).cuda(), torch.randn(T, top, generator=g).cuda(), normal(g, T, K).cuda()

    def steps(stream=None):
        s = mx.moe_sort(ex, E, align=16, stream=stream)
        xs = mx.moe_gather(x, s["slots"], top, stream=stream)
        out = mx.moe_combine(xs, wt, s["pos"], stream=stream)
        b = mx.moe_combine_backward(dout, xs, wt, pos=s["pos"], slots=s["slots"], stream=stream)
        return s | b | dict(xs=xs, out=out)

    a = steps()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = steps(side)
    side.synchronize()
    for k in a:
        assert torch.equal(a[k], c[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps()
    for seed in (2, 3, 4):
        ex.copy_(experts_of(seed, T, top, E, none=0.2))
        x.copy_(normal(generator(seed), T, K))
        graph.replay()
        torch.cuda.synchronize()
        want = steps()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), (seed, k)
