"""The router of many tokens, which takes other kernels than that of few: the same
experts for the same logits, weights, scores and gradients within the roundings of
both (those of few tokens are compared with 64 bits elsewhere)."""
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from layer_util import generator, outs

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
HALF = 2.0 ** -24
FEW, TIMES = 67, 31            # 2077 tokens; each token in every place of a wave's four


def tokens(g, E, dtype):
    """Ordinary logits, masked ones, rows without any, ties, NaN and extreme ones."""
    l = torch.randn(FEW, E, generator=g) * 2
    l[20:30][torch.rand(10, E, generator=g) < 0.8] = float("-inf")
    l[30] = float("-inf")
    l[31] = float("-inf")
    l[31, E - 1] = -3.0
    l[32] = 0.0
    l[33] = torch.arange(E) // 2 % 3
    l[34, 0::2] = -0.0
    l[35] = 50.0
    l[36] = -3.4e38
    l[37] = torch.linspace(-200, 200, E)
    l[38, E // 2] = float("nan")
    l[39] = float("nan")
    l[40:45] = torch.randn(5, E, generator=g) * 1e-7
    return l.to(dtype)


def biases(g, E):
    b = torch.randn(E, generator=g) * 0.1
    yield None
    yield b
    c = b.clone()
    c[::5] = float("-inf")
    yield c
    c = b.clone()
    c[E // 3] = float("inf")
    yield c
    yield b * 1e30
    yield torch.zeros(E)


def same(few, many, tol, what):
    few = few.repeat(TIMES, 1).double()
    many = many.double()
    assert torch.equal(few.isnan(), many.isnan()), what
    few, many = few.nan_to_num(0.0), many.nan_to_num(0.0)
    assert bool(((few - many).abs() <= tol * few.abs() + 2.0 ** -147).all()), what


@pytest.mark.parametrize("E,top,groups,kept", [
    (1, 1, 1, 1), (5, 3, 1, 1), (8, 2, 4, 2), (16, 16, 16, 5), (16, 4, 2, 1), (31, 6, 1, 1), (32, 8, 4, 2),
    (40, 5, 4, 2), (64, 6, 8, 3), (64, 33, 16, 9), (96, 8, 1, 1), (96, 8, 3, 2), (128, 8, 8, 4),
    (160, 6, 5, 3), (200, 64, 1, 1), (256, 8, 8, 4), (256, 40, 16, 7), (256, 8, 2, 1), (256, 3, 64, 9),
    (300, 4, 5, 2)])
def test_many_tokens(E, top, groups, kept):
    g = generator(E * 7 + top)
    # the scores: exponentials and sums of up to E / 16 + 4 terms, on both sides
    tol = 2 * (12 + -(-E // 16) + 4) * HALF
    for dtype in (F32, BF16):
        l = tokens(g, E, dtype).cuda()
        lm = l.repeat(TIMES, 1)
        T = lm.shape[0]
        for bias in biases(g, E):
            b = None if bias is None else bias.cuda()
            for flags in (0, mx.ROUTE_SIGMOID, mx.ROUTE_RENORM | mx.ROUTE_GROUP_PAIR,
                          mx.ROUTE_SIGMOID | mx.ROUTE_RENORM | mx.ROUTE_GROUP_PAIR):
                kw = dict(bias=b, flags=flags, groups=groups, top_groups=kept, scale=2.5, want_scores=True)
                few = mx.moe_route(l, top, **kw)
                buf, broken = outs(dict(experts=((T, top), I32), weights=((T, top), F32), scores=((T, E), F32)))
                many = mx.moe_route(lm, top, out=buf, **kw)
                torch.cuda.synchronize()
                assert broken() == []
                assert torch.equal(few["experts"].repeat(TIMES, 1), many["experts"]), (flags, bias is None)
                same(few["scores"], many["scores"], tol, "scores")
                same(few["weights"], many["weights"], 2 * tol + 2 * (top + 2) * HALF, "weights")


@pytest.mark.parametrize("E,top", [(1, 1), (5, 3), (16, 16), (31, 6), (64, 8), (64, 40), (96, 8), (128, 8),
                                   (256, 8), (300, 20)])
@pytest.mark.parametrize("flags", [0, 1, 2, 3])
def test_many_gradients(E, top, flags):
    g = generator(E * 5 + top + flags)
    for dtype in (F32, BF16):
        l = tokens(g, E, dtype)
        ex = torch.randint(-1, E + 1, (FEW, top), generator=g, dtype=I32)
        dw, ds = torch.randn(FEW, top, generator=g), torch.randn(FEW, E, generator=g)
        for scores in (None, ds):
            def grad(n, out=None):
                r = lambda t: t.repeat(n, 1).cuda()
                return mx.moe_route_backward(r(dw), r(l), r(ex), flags=flags, scale=1.5, out=out,
                                             dscores=None if scores is None else r(scores))
            few = grad(1)
            buf, broken = outs(dict(out=((FEW * TIMES, E), dtype)))
            many = grad(TIMES, buf["out"])
            torch.cuda.synchronize()
            assert broken() == []
            a, b = few.repeat(TIMES, 1).double(), many.double()
            assert torch.equal(a.isnan(), b.isnan())
            a, b = a.nan_to_num(0.0, 0.0, 0.0), b.nan_to_num(0.0, 0.0, 0.0)
            # terms that may cancel: 1.5 dw (over the chosen sum, at least the smallest
            # p chosen, with RENORM) and ds, each with some 40 roundings on either side
            p = torch.sigmoid(l.double()) if flags & 1 else torch.softmax(l.double(), 1)
            p = p.nan_to_num(0.0)
            live = (ex >= 0) & (ex < E)
            w = torch.where(live, dw.double().abs() * 1.5, 0.0)
            chosen = torch.where(live, p.gather(1, ex.clamp(0, E - 1).long()), 0.0)
            s = chosen.sum(1, keepdim=True) if flags & 2 else torch.ones(FEW, 1, dtype=torch.float64)
            part = torch.where(s > 0, w.sum(1, keepdim=True) * 2 / s, 0.0)
            mag = part + (0.0 if scores is None else ds.double().abs())
            bound = p * (mag + (p * mag).sum(1, keepdim=True))
            tol = 2 * (60 + -(-E // 16) + top) * HALF
            half = 2.0 ** -8 if dtype == BF16 else HALF
            limit = (tol * bound).repeat(TIMES, 1).cuda() + 2 * half * a.abs() + 1e-36
            assert bool(((a - b).abs() <= limit).all())
