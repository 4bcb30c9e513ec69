"""NVFP4 matrix-vector products by each kernel and form (product_cases): tokens that fill
its tile and not, several stages of k, odd k and rows, both output types.  Exact
operands as in test_gpu_matvec, whose sums are exact in fp32: at most 9001 products
that are multiples of 1/16 and add to less than 2^24 of them (checked)."""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from product_cases import EXPERTS, MATVEC
from product_util import Guarded, assert_equal, nv_values, product, to_dev
from test_gpu_matvec import DT, dev, exact_tokens, exact_weight, experts_want, sg_of, values

pytestmark = pytest.mark.gpu


def assert_exact_in_fp32(x):
    """Weights (before the tensor scale) are at most 6 * 2."""
    assert np.abs(values(x)).sum(axis=1).max() * 12 * 16 < 2 ** 24


@pytest.mark.parametrize("T,N,K", [s for s, _ in MATVEC])
def test_matvec(T, N, K):
    x, (q, s) = exact_tokens(T, K, T + N), exact_weight(N, K, N + K)
    want = product(values(x), nv_values(q, s, 0.125, N, K))[0]
    assert_exact_in_fp32(x)
    for out in (0, mx.OUT_F32):
        y = Guarded((T, N), DT[out])
        mx.nvfp4_matvec(to_dev(x), dev(q), dev(s), sg_of(0.125), flags=out, out=y.t)
        torch.cuda.synchronize()
        y.check("matvec")
        assert_equal(y.t, want, f"{T} {N} {K} {out}")


@pytest.mark.parametrize("T,top,G,N,K", [s for s, _ in EXPERTS])
def test_experts(T, top, G, N, K):
    """Slots with repeated experts and without one; then all of one expert, more slots
    than its kernel takes at a time."""
    rng = np.random.default_rng(T + N)
    x, (q, s) = exact_tokens(T, K, 1), exact_weight(G * N, K, 2)
    assert_exact_in_fp32(x)
    sg = [2.0 ** -(g % 5) for g in range(G)]
    mixed = rng.integers(0, G, size=(T, top)).astype(np.int32)
    mixed[rng.random((T, top)) < 0.2] = -1
    for e in (mixed, np.full((T, top), G - 1, np.int32)):
        want = experts_want(x, e, q, s, sg, N, K)[0]
        for out in (0, mx.OUT_F32):
            y = Guarded((T, top, N), DT[out])
            mx.nvfp4_matvec_experts(to_dev(x), dev(e), dev(q), dev(s), sg_of(*sg), flags=out, out=y.t)
            torch.cuda.synchronize()
            y.check("experts")
            assert_equal(y.t, want, f"{T} {top} {G} {out}")
