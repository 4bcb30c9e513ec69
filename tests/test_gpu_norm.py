"""The root-mean-square norm and its gradients against 64 bits: h to the bit, the
casts byte for byte against the oracle's casts of the norm's own bf16 output, the
rest within bounds derived from the sums' lengths.

Rounding of a sum of positive terms: a term passes through at most `chain` fp32
additions, each off by 2^-24 of what it adds up to, so the sum is off by at most
chain 2^-24 of itself.  A row in registers adds 16 elements in two chains of 8 (with
their squares' exact product inside the FMA), 1, 6 steps over the wave and up to
15 over the waves: 30.  A longer one is added by 512 threads, 8 of every 4096 each in
a line, then 6 steps and 8."""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
import oracle as O
from gpu_util import assert_same
from layer_util import f64, generator, host_bits, normal, outs

pytestmark = pytest.mark.gpu

U8, F32, BF16 = torch.uint8, torch.float32, torch.bfloat16
HALF = 2.0 ** -24          # half a step of fp32, relative
EPS = 1e-5


def chain(K):
    return 30 if K <= 16384 else 8 * -(-K // 4096) + 15


def spec(M, K, axis, residual, y, ckpt):
    need = dict(rstd=((M,), F32))
    if residual:
        need["h"] = ((M, K), BF16)
    if y:
        need["y"] = ((M, K), BF16)
    for bit, name, r, c in ((1, "row", M, K), (2, "col", K, M)):
        if axis & bit:
            need["q_" + name] = ((r, c), U8)
            need["s_" + name] = ((max(1, mx.mx_scale_size(r, c, axis)),), U8)
    if ckpt:
        need["q_h"] = ((M, K), U8)
        need["s_h"] = ((M, -(-K // 32)), U8)
    return need


def check_norm(x, w, res, axis=0, eps=EPS, ckpt=False):
    M, K = x.shape
    buf, broken = outs(spec(M, K, axis, res is not None, True, ckpt))
    dev = lambda t: None if t is None else t.cuda()
    o = mx.mx_rmsnorm(dev(x), dev(w), residual=dev(res), eps=eps, axis=axis, want_y=True,
                      checkpoint=ckpt, out=buf)
    torch.cuda.synchronize()
    assert broken() == []
    h = x if res is None else (x.float() + res.float()).to(BF16)
    assert_same(host_bits(o["h"]), host_bits(h), "h")
    hd = f64(h)
    rstd = ((hd * hd).mean(1) + np.float32(eps).astype(np.float64)) ** -0.5
    # 64 bits, rounded once
    tol = 1.001 * HALF
    got = f64(o["rstd"])
    assert np.all(np.abs(got - rstd) <= tol * rstd), np.max(np.abs(got / rstd - 1)) / HALF
    # 64 bits, rounded to fp32 and then to bf16 (an element whose rounding to fp32 the
    # last bits of 64 turn over, and that is half way between two bf16 as well, would
    # differ: one of 2^38)
    y = torch.from_numpy(hd * rstd[:, None] * (1.0 if w is None else f64(w)))
    assert_same(host_bits(o["y"]), host_bits(y.float().to(BF16)), "y")
    if axis:
        assert_same_casts(o, host_bits(o["y"]), axis)
    if ckpt:
        c = O.mx_quantize(host_bits(o["h"]), axis=1 | mx.SCALE_ROUND_UP)
        assert_same(o["q_h"], c["q_row"], "q_h")
        assert_same(o["s_h"], c["s_row"], "s_h")
    return o


def assert_same_casts(o, y, axis):
    want = O.mx_quantize(y, axis=axis)
    for k in ("q_row", "s_row", "q_col", "s_col"):
        if want.get(k) is not None:
            got = o[k].cpu().numpy().reshape(-1)
            assert_same(got, np.asarray(want[k]).reshape(-1), k)


SIZES = [(1, 1), (1, 8), (3, 32), (5, 40), (7, 31), (2, 511), (33, 512), (17, 520), (64, 1024),
         (31, 4096), (130, 1111), (16, 16384), (3, 16392), (5, 20001), (1, 8192), (300, 256),
         (2, 16383), (257, 96), (1040, 136), (48, 7168)]


@pytest.mark.parametrize("M,K", SIZES)
def test_norm(M, K):
    g = generator(M * 7 + K)
    x, w, res = normal(g, M, K), normal(g, K), normal(g, M, K, scale=3.0)
    check_norm(x, w, res)
    check_norm(x, None, None, axis=1, ckpt=True)
    check_norm(x, w, res, axis=3, ckpt=True)
    check_norm(x, w, None, axis=2 | mx.SCALE_TILED | mx.ELEM_E5M2)
    check_norm(x, w, res, axis=3 | mx.SCALE_TILED | mx.SCALE_ROUND_UP)
    check_norm(x, None, res, axis=3 | mx.ELEM_E5M2 | mx.SCALE_ROUND_UP)


@pytest.mark.parametrize("first", [1, 4089, 8193, 16385])
def test_every_end_of_a_row(first):
    """Row lengths of every remainder mod 8, in each kind of kernel, forward and back."""
    for K in range(first, first + (24 if first == 1 else 8)):
        g = generator(K)
        dy, x, w, res = normal(g, 3, K), normal(g, 3, K), normal(g, K), normal(g, 3, K)
        check_norm(x, w, res, axis=3, ckpt=True)
        check_back(dy, x, w, res)
        check_back(dy, x, w, res, ckpt=True)


@pytest.mark.parametrize("M,K", [(16411, 1024), (16384, 1032)])
def test_norm_of_many_rows(M, K):
    """Two rows a workgroup, a few of them none."""
    g = generator(M + K)
    x, w, res = normal(g, M, K), normal(g, K), normal(g, M, K, scale=3.0)
    check_norm(x, w, res, axis=3 | mx.SCALE_TILED, ckpt=True)
    check_norm(x, w, None, axis=1)


def test_norm_without_y_gives_the_same_casts():
    g = generator(1)
    for M, K in ((96, 1000), (37, 77)):
        x, w, res = normal(g, M, K).cuda(), normal(g, K).cuda(), normal(g, M, K).cuda()
        a = mx.mx_rmsnorm(x, w, residual=res, axis=3, want_y=True)
        b = mx.mx_rmsnorm(x, w, residual=res, axis=3)
        assert b["y"] is None and b["q_h"] is None
        for k in ("h", "rstd", "q_row", "s_row", "q_col", "s_col"):
            assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("K", [256, 100])
def test_norm_of_special_rows(K):
    """Zeros, Inf, NaN, the largest and the smallest numbers stay in their rows."""
    g = generator(K)
    x = normal(g, 12, K)
    clean = mx.mx_rmsnorm(x.cuda(), eps=EPS, axis=1)
    x[1] = 0
    x[3, 5] = float("inf")
    x[5, K - 1] = float("nan")
    x[7] = 3e38
    x[9] = 1e-40
    o = mx.mx_rmsnorm(x.cuda(), eps=EPS, axis=1, want_y=True)
    torch.cuda.synchronize()
    y, rstd = f64(o["y"]), f64(o["rstd"])
    assert np.all(y[1] == 0) and abs(rstd[1] * EPS ** 0.5 - 1) < 1e-6
    assert rstd[3] == 0 and np.isnan(y[3, 5]) and np.all(y[3, :5] == 0)
    assert np.isnan(rstd[5]) and np.isnan(y[5]).all()
    assert np.all(y[7] == 1.0)                          # squares past fp32
    assert np.isfinite(y[9]).all()
    assert_same_casts(o, host_bits(o["y"]), 1)
    for r in (0, 2, 4, 6, 8, 10, 11):
        assert torch.equal(o["q_row"][r], clean["q_row"][r]), r


# ---- gradients -----------------------------------------------------------------

def check_back(dy, x, w, dres, ckpt=False, eps=EPS):
    M, K = x.shape
    f = mx.mx_rmsnorm(x.cuda(), None if w is None else w.cuda(), eps=eps, checkpoint=ckpt)
    h = f64(x)
    src = dict(h=f["h"])
    if ckpt:
        src = dict(q_h=f["q_h"], s_h=f["s_h"])
        q = f["q_h"].cpu().view(torch.float8_e4m3fn).double().numpy()
        h = q * np.repeat(np.exp2(f64(f["s_h"]) - 127), 32, axis=1)[:, :K]
    buf, broken = outs(dict(dh=((M, K), BF16), dweight=((K,), F32)))
    dev = lambda t: None if t is None else t.cuda()
    o = mx.mx_rmsnorm_backward(dy.cuda(), f["rstd"], dev(w), dres=dev(dres), out=buf, **src)
    torch.cuda.synchronize()
    assert broken() == []
    rstd, d = f64(f["rstd"])[:, None], f64(dy)
    xh, gw = h * rstd, d * (1.0 if w is None else f64(w))
    c = (gw * xh).mean(1, keepdims=True)
    r = 0.0 if dres is None else f64(dres)
    dh = r + rstd * (gw - xh * c)
    # c: 3 roundings of each term (g, xhat, and the mean), `chain` of the sum
    ec = (chain(K) + 4) * HALF * np.abs(gw * xh).mean(1, keepdims=True)
    inner = rstd * (2 * HALF * np.abs(gw) + 4 * HALF * np.abs(xh * c) + np.abs(xh) * ec)
    bound = 2.0 ** -8 * np.abs(dh) + 1.01 * (inner + 3 * HALF * (np.abs(dh) + np.abs(r))) + 1e-38
    assert np.all(np.abs(f64(o["dh"]) - dh) <= bound)
    # a workgroup adds its rows in a line (with at least min(M, 64) of them), 32
    # slices add the workgroups' (at most 512) and one thread the slices
    dw, mag = (d * xh).sum(0), np.abs(d * xh).sum(0)
    adds = -(-M // min(M, 64)) + 16 + 32 + 1
    assert np.all(np.abs(f64(o["dweight"]) - dw) <= adds * HALF * mag + 1e-38)
    return o


@pytest.mark.parametrize("M,K", SIZES + [(700, 64), (1500, 1024), (2001, 72), (513, 20)])
def test_norm_backward(M, K):
    g = generator(M * 11 + K)
    dy, x, w, dres = normal(g, M, K), normal(g, M, K, scale=2.0), normal(g, K), normal(g, M, K)
    check_back(dy, x, w, dres)
    check_back(dy, x, None, None)
    check_back(dy, x, w, dres, ckpt=True)


def test_norm_backward_without_dweight():
    g = generator(3)
    for M, K in ((40, 512), (9, 33)):
        dy, x, w = normal(g, M, K).cuda(), normal(g, M, K).cuda(), normal(g, K).cuda()
        f = mx.mx_rmsnorm(x, w)
        a = mx.mx_rmsnorm_backward(dy, f["rstd"], w, h=x)
        b = mx.mx_rmsnorm_backward(dy, f["rstd"], w, h=x, want_dweight=False)
        assert b["dweight"] is None and torch.equal(a["dh"], b["dh"])


@pytest.mark.parametrize("K", [256, 100])
def test_norm_backward_of_special_rows(K):
    """A row that holds Inf or NaN has NaN gradients, from bf16 and from the 8-bit copy,
    and leaves the other rows' alone."""
    g = generator(K)
    x, dy = normal(g, 9, K), normal(g, 9, K)
    def grads(x, **src):
        f = mx.mx_rmsnorm(x.cuda(), eps=EPS, checkpoint=True)
        a = mx.mx_rmsnorm_backward(dy.cuda(), f["rstd"], h=f["h"])["dh"]
        b = mx.mx_rmsnorm_backward(dy.cuda(), f["rstd"], q_h=f["q_h"], s_h=f["s_h"])["dh"]
        return a, b
    clean = grads(x)
    x[2, K - 1] = float("nan")
    x[5, 0] = float("nan")
    for a, c in zip(grads(x), clean):
        assert bool(a[2].isnan().all()) and bool(a[5].isnan().all())
        for r in (0, 1, 3, 4, 6, 7, 8):
            assert torch.equal(a[r], c[r]), r


def same_rows(M, K, **kw):
    """The last rows of a tensor past 2^31 elements against the same rows alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    n = 64
    x = torch.empty(M, K, dtype=BF16, device="cuda")
    x[-n:] = torch.randn(n, K, generator=g, device="cuda").to(BF16)
    x[:-n] = 1.0
    return x, n


def test_norm_past_32_bit_offsets():
    """2^31 elements and more, with every output: the last rows as when they are alone,
    and the last row blocks of the column-wise cast likewise."""
    M, K = 262208, 8200             # 2.15e9 elements, a multiple of 32 rows
    x, n = same_rows(M, K)
    w = torch.linspace(0.5, 2.0, K, device="cuda").to(BF16)
    o = mx.mx_rmsnorm(x, w, axis=3, want_y=True, checkpoint=True)
    tail = x[-n:].clone()
    t = mx.mx_rmsnorm(tail, w, axis=3, want_y=True, checkpoint=True)
    for k in ("y", "rstd", "q_row", "s_row", "q_h", "s_h"):
        assert torch.equal(o[k][-n:], t[k]), k
    assert torch.equal(o["q_col"][:, -n:], t["q_col"]) and torch.equal(o["s_col"][:, -2:], t["s_col"])
    del o["q_col"], o["q_row"], o["y"]
    dy = torch.zeros_like(x)
    dy[-n:] = tail.flip(0)
    a = mx.mx_rmsnorm_backward(dy, o["rstd"], w, q_h=o["q_h"], s_h=o["s_h"])
    b = mx.mx_rmsnorm_backward(dy[-n:].clone(), t["rstd"], w, q_h=t["q_h"], s_h=t["s_h"])
    assert torch.equal(a["dh"][-n:], b["dh"]) and not bool(a["dh"][:-n].any())
    # zeros, and the same 64 rows in other workgroups: fp32 sums of 64 terms
    mag = (dy[-n:].float() * tail.float() * t["rstd"][:, None]).abs().sum(0)
    assert bool(((a["dweight"] - b["dweight"]).abs() <= 128 * HALF * mag + 1e-38).all())


@pytest.mark.parametrize("K", [24, 15])
def test_norm_backward_against_differences(K):
    """dh and dweight against central differences of sum(dy y) in 64 bits: the
    difference quotient of a function whose third derivative is d3 is off by
    step^2 / 6 d3, here below 1e-7, and by rounding 1e-16 / step, below 1e-9."""
    M, g, step = 3, generator(5), 1e-5
    dy, x, w = normal(g, M, K), normal(g, M, K), normal(g, K)
    o = check_back(dy, x, w, None)
    d, h, wd = f64(dy), f64(x), f64(w)

    def loss(h, wd):
        return (d * h * ((h * h).mean(1, keepdims=True) + np.float64(np.float32(EPS))) ** -0.5 * wd).sum()

    for m in range(M):
        for k in range(K):
            e = np.zeros_like(h)
            e[m, k] = step
            num = (loss(h + e, wd) - loss(h - e, wd)) / (2 * step)
            assert abs(f64(o["dh"])[m, k] - num) <= 2.0 ** -8 * abs(num) + 1e-5
    for k in range(K):
        e = np.zeros_like(wd)
        e[k] = step
        num = (loss(h, wd + e) - loss(h, wd - e)) / (2 * step)
        assert abs(f64(o["dweight"])[k] - num) <= 1e-5


# ---- streams, graphs, repeats ----------------------------------------------------

def both(x, w, res, dy, stream=None, bufs=None):
    a, b = bufs or (None, None)
    f = mx.mx_rmsnorm(x, w, residual=res, axis=3, checkpoint=True, out=a, stream=stream)
    r = mx.mx_rmsnorm_backward(dy, f["rstd"], w, q_h=f["q_h"], s_h=f["s_h"], dres=res, out=b,
                               stream=stream)
    return {k: v for k, v in (f | r).items() if v is not None}


def inputs(M, K, seed):
    g = generator(seed)
    return [t.cuda() for t in (normal(g, M, K), normal(g, K), normal(g, M, K), normal(g, M, K))]


@pytest.mark.parametrize("M,K", [(600, 2048), (100, 301)])
def test_norm_is_the_same_each_time_and_on_any_stream(M, K):
    t = inputs(M, K, 8)
    a = both(*t)
    b = both(*t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = both(*t, stream=s)
    s.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


@pytest.mark.parametrize("M,K", [(600, 2048), (100, 301)])
def test_norm_in_a_graph(M, K):
    t = inputs(M, K, 9)
    both(*t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(*t)
    for seed in (10, 11, 12):
        new = inputs(M, K, seed)
        for old, v in zip(t, new):
            old.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = both(*new)
        for k in want:
            assert torch.equal(got[k], want[k]), (seed, k)
