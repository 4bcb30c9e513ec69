"""The norm at the ends of the numbers' range, against 64 bits to the bit: finite rows
and weights whose product passes fp32, or falls below what fp32 holds, while the output
does not, in each kernel, with the casts of that output against the oracle."""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from gpu_util import assert_same
from layer_util import f64, generator, host_bits, normal, outs
from test_gpu_norm import HALF, assert_same_casts, spec

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# one and two chunks a lane, whole and not, read twice, whole and not
SIZES = [(37, 264), (5, 77), (40, 1000), (130, 1111), (16, 7168), (33, 9001), (3, 16392), (3, 16391), (300, 128)]
AXES = (0, 1, 3, 2 | mx.SCALE_TILED)


def check(x, w, eps=0.0, residual=None):
    """y to the bit: 64 bits rounded to fp32 and then to bf16; NaN where that is."""
    M, K = x.shape
    h = x if residual is None else (x.float() + residual.float()).to(BF16)
    hd, wd = f64(h), f64(w)
    with np.errstate(all="ignore"):
        rstd = ((hd * hd).mean(1) + np.float64(np.float32(eps))) ** -0.5
        want = torch.from_numpy(hd * wd * rstd[:, None]).float().to(BF16)
    nan = want.isnan()
    for axis in AXES:
        buf, broken = outs(spec(M, K, axis, residual is not None, True, False))
        o = mx.mx_rmsnorm(x.cuda(), w.cuda(), residual=None if residual is None else residual.cuda(), eps=eps,
                          axis=axis, want_y=True, out=buf)
        torch.cuda.synchronize()
        assert broken() == []
        y = o["y"].cpu()
        assert torch.equal(y.isnan(), nan)
        assert_same(host_bits(y.masked_fill(nan, 0.0)), host_bits(want.masked_fill(nan, 0.0)), "y")
        if axis:
            assert_same_casts(o, host_bits(o["y"]), axis)
        got = f64(o["rstd"])
        ok = np.isfinite(rstd)
        assert np.all(np.abs(got[ok] - rstd[ok]) <= 1.001 * (HALF * rstd[ok] + 2.0 ** -150))
    return want


def logs(g, lo, hi, *shape):
    """Powers of two of both signs, a few bits beside them."""
    v = torch.exp2(torch.randint(lo, hi + 1, shape, generator=g).double())
    v = v * (1 + torch.randint(0, 128, shape, generator=g) / 128) * (1 - 2 * torch.randint(0, 2, shape, generator=g))
    return v.clamp(-3.38e38, 3.38e38).to(BF16)


@pytest.mark.parametrize("M,K", SIZES)
def test_rows_of_the_largest_numbers(M, K):
    g = generator(M + K)
    w = 1.25 + 2.75 * torch.rand(K, generator=g)
    for x in (torch.full((M, K), 3e38), torch.full((M, K), 2.0 ** 127),
              normal(g, M, K).float().clamp(-4, 4) * 2.0 ** 125):
        y = check(x.to(BF16), w.to(BF16))
        assert bool(y.isfinite().all())
    # among them rows of ordinary numbers, and with an eps and a residual
    x = normal(g, M, K)
    x[::3] = torch.tensor(3e38)
    assert bool(check(x, w.to(BF16), eps=1e-5).isfinite().all())
    r = normal(g, M, K)
    r[1::3] = torch.tensor(-2e38)
    assert bool(check(x, w.to(BF16), eps=1e-5, residual=r).isfinite().all())


@pytest.mark.parametrize("M,K", SIZES)
def test_rows_and_weights_of_tiny_numbers(M, K):
    g = generator(M * K)
    tiny = normal(g, M, K).float()
    for h, wt in ((1e-36, 1e-8), (1e-30, 1e-12), (1e-20, 1e-25), (2.0 ** -120, 2.0 ** -20), (1e-38, 3.0)):
        w = (wt * (1 + torch.rand(K, generator=g))).to(BF16)
        y = check((tiny * h).to(BF16), w)
        assert bool((y != 0).float().mean() > 0.9)
    x = tiny.to(BF16)
    x[::2] = (tiny[::2] * 1e-35).to(BF16)
    check(x, (1e-9 * torch.rand(K, generator=g)).to(BF16))


@pytest.mark.parametrize("M,K", SIZES)
def test_ordinary_rows_by_weights_of_any_size(M, K):
    g = generator(M * 3 + K)
    x = normal(g, M, K, scale=2.0 ** 30)
    check(x, logs(g, 90, 120, K))
    check(x, logs(g, -100, 100, K))
    w = normal(g, K)
    w[K // 2] = torch.tensor(2.0 ** 127)
    w[K // 3] = torch.tensor(-2.0 ** -130)
    w[K // 4] = 0
    check(normal(g, M, K), w, eps=1e-5)


@pytest.mark.parametrize("M,K", SIZES)
def test_rows_with_inf_beside_large_weights(M, K):
    """rstd is 0: zeros with the products' signs, though the products pass fp32, and NaN
    in the Inf's own place."""
    g = generator(M + 5 * K)
    x, w = logs(g, 100, 127, M, K), logs(g, 60, 127, K)
    x[:, K // 2] = float("inf")
    y = check(x, w)
    assert bool(y[:, K // 2].isnan().all()) and int(y.isnan().sum()) == M


@pytest.mark.parametrize("K", [264, 1111, 16392])
def test_rows_of_each_magnitude(K):
    """A row for each power of two that bf16's normal numbers have, by weights of 1 and by
    such as pass fp32 with the first and the last of them."""
    g = generator(K)
    x = normal(g, 250, K).float().clamp(-3.9, 3.9) * torch.exp2(torch.arange(250.0) - 124).view(-1, 1)
    for w in (torch.ones(K), 1.5 * torch.ones(K), 2.0 ** 60 * torch.ones(K), 2.0 ** -60 * torch.ones(K)):
        check(x.clamp(-3.3e38, 3.3e38).to(BF16), w.to(BF16))


@pytest.mark.parametrize("K", [264, 77, 1111, 16392])
def test_one_row_of_the_largest_numbers_anywhere(K):
    """One row among ordinary ones, in each place of a tile and a half of 128 rows: as it
    is alone, the others as without it, columns as mx_quantize casts that y."""
    g = generator(K)
    M = 200
    x, w = normal(g, M, K).cuda(), (1.25 + torch.rand(K, generator=g)).to(BF16).cuda()
    clean = mx.mx_rmsnorm(x, w, axis=3, want_y=True)
    rows = [r for r in range(M) if r % 3 == 0 or r % 32 in (15, 16, 31)] if K > 2000 else range(M)
    for r in rows:
        z = x.clone()
        z[r] *= 2.0 ** 125
        a = mx.mx_rmsnorm(z, w, axis=3, want_y=True)
        b = mx.mx_rmsnorm(z[r:r + 1].clone(), w, axis=1, want_y=True)
        assert torch.equal(a["y"][r], b["y"][0]) and bool(a["y"][r].isfinite().all()), r
        rest = torch.arange(M, device="cuda") != r
        assert torch.equal(a["y"][rest], clean["y"][rest]), r
        assert torch.equal(a["q_row"][rest], clean["q_row"][rest]), r
        c = mx.mx_quantize(a["y"], axis=2)
        assert torch.equal(a["q_col"], c["q_col"]) and torch.equal(a["s_col"], c["s_col"]), r
