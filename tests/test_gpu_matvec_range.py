"""NVFP4 matrix-vector products at the ends of the tokens' range and at fp32's last bit.

The sums hold in fp32's range and no partial sum of scaled products leaves it, so
every number of tokens has to give the 64-bit product within product_util's
tolerance; sums of multiples of 2^-8 below 2^16 are exact in fp32 in any order and
have to be equal to it.
"""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
import workloads as W
from product_util import E4M3, assert_close, assert_equal, nv_values, product, to_dev
from test_gpu_matvec import dev, experts_want, sg_of, values

pytestmark = pytest.mark.gpu

TOKENS = [1, 2, 3, 17]


def code(v):
    return int(np.flatnonzero(E4M3 == v)[0])


def weight(N, K, scales, seed):
    """Random codes; block scales drawn from `scales`, either sign."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, size=(N, -(-K // 2))).astype(np.uint8)
    if K % 2:
        q[:, -1] &= 15
    s = np.array([code(v) for v in scales], np.uint8)[rng.integers(0, len(scales), size=(N, -(-K // 16)))]
    return q, s | (rng.integers(0, 2, size=s.shape) << 7).astype(np.uint8)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("K", [32, 700])
def test_largest_tokens_with_small_block_scales(T, K):
    """|x| up to bf16's largest in one block, scales of 2^-9 .. 2^-6: 16 products of at
    most 6 * 2^-6 of it."""
    N = 96
    rng = np.random.default_rng(T + K)
    q, s = weight(N, K, [2. ** -9, 3 * 2. ** -9, 2. ** -7, 2. ** -6], 1)
    x = np.zeros((T, K), np.uint16)
    x[:, 16:32] = 0x7F00 + rng.integers(0, 0x80, size=(T, 16)) + 0x8000 * rng.integers(0, 2, size=(T, 16))
    x[:, 0] = 0x3F80
    v = nv_values(q, s, 1.0, N, K)
    want, mag = product(values(x), v)
    assert mag.max() < 3.3e38 and np.abs(6 * values(x)).max() > 3.5e38
    for flags in (0, mx.OUT_F32):
        y = mx.nvfp4_matvec(to_dev(x), dev(q), dev(s), sg_of(1.0), flags=flags)
        assert_close(y, want, mag, K + 1, f"{T} {K} {flags}")
        e = np.full((T, 1), 1, np.int32)
        y = mx.nvfp4_matvec_experts(to_dev(x), dev(e), dev(np.concatenate([q, q])),
                                    dev(np.concatenate([s, s])), sg_of(0.0, 1.0), flags=flags)
        assert_close(y, want[:, None], mag[:, None], K + 1, f"experts {T} {K} {flags}")


@pytest.mark.parametrize("T", TOKENS)
def test_subnormal_tokens(T):
    """bf16's subnormal numbers, times scales of 2^5 .. 448: nothing is flushed.  One
    product an output, exact in fp32."""
    N, K = 64, 256
    q, s = weight(N, K, [32., 448.], 2)
    x = np.zeros((T, K), np.uint16)
    rng = np.random.default_rng(T)
    x[np.arange(T), rng.integers(0, K, size=T)] = rng.integers(1, 0x80, size=T)
    want = product(values(x), nv_values(q, s, 1.0, N, K))[0]
    y = mx.nvfp4_matvec(to_dev(x), dev(q), dev(s), sg_of(1.0), flags=mx.OUT_F32)
    assert bool((y != 0).any())
    assert_equal(y, want, f"subnormal {T}")


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("K", [64, 4095])
def test_sums_of_24_bits(T, K):
    """A product of 2^15 and multiples of 2^-8 that add to less than 2^15."""
    N = 80
    rng = np.random.default_rng(T + K)
    q, s = weight(N, K, [0.25, 0.5, 1.0], 3)
    xf = rng.integers(-8, 9, size=(T, K)).astype(np.float32) * 2.0 ** -5    # codes 2^-1, scales 2^-2
    at = K // 3
    xf[:, at] = 2.0 ** 14
    q[:, at // 2] = 0x22                                    # both codes 1
    s[:, at // 16] = code(1.0)
    x = W.bf16_bits(xf)
    v = nv_values(q, s, 1.0, N, K)
    want, mag = product(values(x), v)
    assert mag.max() < 2.0 ** 16 and np.abs(want).max() > 2.0 ** 13
    y = mx.nvfp4_matvec(to_dev(x), dev(q), dev(s), sg_of(1.0), flags=mx.OUT_F32)
    assert_equal(y, want, f"24 bits {T} {K}")
