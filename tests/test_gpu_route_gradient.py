"""The gradient of normalised weights where it cancels: exactly 0 for a token with one
live choice, and right to a few roundings of itself where one choice outweighs the rest
or all scores are tiny."""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from layer_util import f64, generator

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
HALF = 2.0 ** -24
SOFTMAX, SIGMOID = mx.ROUTE_RENORM, mx.ROUTE_RENORM | mx.ROUTE_SIGMOID
LOW = float("-inf")


@pytest.mark.parametrize("flags", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [1, 8, 20, 64, 100, 256, 600])
@pytest.mark.parametrize("T", [5, 2048, 2049, 3001])
def test_one_live_choice_has_no_gradient(flags, E, T):
    g = generator(T + E)
    for dtype in (F32, BF16):
        l = (torch.randn(T, E, generator=g) * 2).to(dtype).cuda()
        one = torch.full_like(l, LOW)
        at = torch.randint(0, E, (T, 1), generator=g).cuda()
        one.scatter_(1, at, l.gather(1, at))
        for x, top in ((l, 1), (one, min(4, E))):
            ex = mx.moe_route(x, top, flags=flags)["experts"]
            assert bool((ex[:, 0] >= 0).all()) and bool((ex[:, 1:] == -1).all())
            dw = torch.randn(T, top, generator=g).cuda()
            o = mx.moe_route_backward(dw, x, ex, flags=flags, scale=2.5)
            assert not bool(o.any()), (top, float(o.abs().max()))
            # the scores' part alone is left
            ds = torch.randn(T, E, generator=g).cuda()
            a = mx.moe_route_backward(dw, x, ex, flags=flags, scale=2.5, dscores=ds)
            b = mx.moe_route_backward(torch.zeros_like(dw), x, ex, flags=flags, scale=2.5, dscores=ds)
            assert torch.equal(a, b)


# With w_i = p_i / sum p: dl_i = w_i (d_i - sum_j w_j d_j) = w_i sum_j w_j (d_i - d_j), d =
# scale dw; by sigmoid times 1 - p_i.  p's roundings (exp 2 ulp, its sum, 1 / sum and the
# product) count relatively, for the formula holds for the rounded p as well: 8 half steps
# of each p, three p in a term; the products and the output a few more.  d is rounded to
# fp32.  What cancels is d_i sp - sd with sp = p_1 + p_2 and sd = d_1 p_1 + d_2 p_2: each
# product of two fp32 numbers is exact in 64 bits, the two sums and the difference are
# rounded, each by 2^-53 of at most (|d_1| + |d_2|) sp: 3 2^-53 (|d_1| + |d_2|) in all,
# after 1 / sp, times w_i.
@pytest.mark.parametrize("flags", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [2, 8, 64, 256])
@pytest.mark.parametrize("T", [33, 2500])
@pytest.mark.parametrize("gap", [5.0, 12.0, 25.0, 60.0])
def test_one_choice_outweighs_the_other(flags, E, T, gap):
    g = generator(E + T)
    l = torch.full((T, E), LOW)
    l[:, 0] = (torch.randn(T, generator=g) * 64).round() / 64 - gap / 2   # differences are exact
    l[:, E - 1] = l[:, 0] + gap
    if flags == SIGMOID:
        l -= gap / 2                     # both below 0, where scores part by the gap
    ex = torch.tensor([[E - 1, 0]], dtype=I32).repeat(T, 1)
    dw = torch.randn(T, 2, generator=g)
    o = f64(mx.moe_route_backward(dw.cuda(), l.cuda(), ex.cuda(), flags=flags, scale=0.75))
    x, d = f64(l[:, [E - 1, 0]]), 0.75 * f64(dw)
    p = 1 / (1 + np.exp(-x)) if flags == SIGMOID else np.exp(x - x.max(1, keepdims=True))
    w = p / p.sum(1, keepdims=True)
    want = w[:, 0] * w[:, 1] * (d[:, 0] - d[:, 1])
    size = np.abs(d).sum(1)
    tol = 1.01 * HALF * (w[:, 0] * w[:, 1] * size) + 32 * HALF * np.abs(want) + 2.0 ** -149
    for col, sign, k in ((E - 1, 1, 0), (0, -1, 1)):
        q = 1 / (1 + np.exp(x[:, k])) if flags == SIGMOID else 1.0
        assert np.all(np.abs(o[:, col] - sign * want * q) <= tol + 3.01 * 2.0 ** -53 * w[:, k] * size), col
    if E > 2:
        assert not o[:, 1:E - 1].any()


@pytest.mark.parametrize("T", [3, 2100])
@pytest.mark.parametrize("at", [-80.0, -89.0, -93.0])
def test_scores_too_small_for_a_reciprocal(at, T):
    """Sigmoid scores near and below fp32's normal numbers, whose sum has no fp32
    reciprocal: the weights and their gradient stay finite.  p is within 2^-150 and 8
    half steps of itself."""
    E = 16
    l = torch.full((T, E), 2 * at)
    l[:, 3], l[:, 9] = at, at - 1
    ex = torch.tensor([[3, 9]], dtype=I32).repeat(T, 1)
    dw = torch.tensor([[1.0, -0.5]]).repeat(T, 1)
    o = f64(mx.moe_route_backward(dw.cuda(), l.cuda(), ex.cuda(), flags=SIGMOID))
    p = np.exp(f64(l[0, [3, 9]]))
    w = p / p.sum()
    want = w[0] * w[1] * 1.5
    tol = (3 * 2.0 ** -150 / p[1] + 40 * HALF) * want
    assert np.all(np.abs(o[:, 3] - want) <= tol) and np.all(np.abs(o[:, 9] + want) <= tol)
