"""NVFP4 matrix-vector products with operands smaller than one load: fewer than 8 token
elements, 16 bytes of codes or 4 of scales, with few and with many outputs (operands
and references: test_gpu_matvec)."""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from product_util import Guarded, assert_equal, nv_values, product, to_dev
from test_gpu_matvec import DT, dev, exact_tokens, exact_weight, experts_want, sg_of, values

pytestmark = pytest.mark.gpu

# few token elements, many rows; few weights, many tokens
SHAPES = [(1, 1, 1), (1, 100003, 7), (7, 70001, 1), (3, 257, 2), (1, 1 << 21, 5), (70001, 1, 15),
          (5000, 31, 1), (300, 3, 16), (40001, 1, 48), (9, 2, 33)]


@pytest.mark.parametrize("out", [0, mx.OUT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_tiny_operands(T, N, K, out):
    x, (q, s) = exact_tokens(T, K, T + N), exact_weight(N, K, N + K)
    y = Guarded((T, N), DT[out])
    mx.nvfp4_matvec(to_dev(x), dev(q), dev(s), sg_of(0.25), flags=out, out=y.t)
    torch.cuda.synchronize()
    y.check("matvec")
    assert_equal(y.t, product(values(x), nv_values(q, s, 0.25, N, K))[0], f"{T} {N} {K}")


@pytest.mark.parametrize("T,top,G,N,K", [(1, 3, 4, 50021, 7), (7, 5, 3, 9001, 1), (2, 64, 9, 1000, 3),
                                         (1, 64, 1, 31, 1), (4000, 3, 2, 1, 15), (50, 2, 1, 1, 47)])
def test_tiny_operands_of_experts(T, top, G, N, K):
    rng = np.random.default_rng(T + N)
    x, (q, s) = exact_tokens(T, K, 1), exact_weight(G * N, K, 2)
    sg = [2.0 ** -g for g in range(G)]
    e = rng.integers(-1, G + 1, size=(T, top)).astype(np.int32)      # -1 and G: no expert
    e[0, 0] = -2 ** 31
    y = Guarded((T, top, N), torch.bfloat16)
    mx.nvfp4_matvec_experts(to_dev(x), dev(e), dev(q), dev(s), sg_of(*sg), out=y.t)
    torch.cuda.synchronize()
    y.check("experts")
    assert_equal(y.t, experts_want(x, e, q, s, sg, N, K)[0], f"{T} {top} {G}")
