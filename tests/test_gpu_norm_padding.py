"""What pads the tile layout of the norm's scales, and the blocks that a tensor ends
inside, is as mx_quantize writes it whatever the rows and the weights hold: NaN, Inf,
zeros without an eps, weights of Inf and NaN."""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from layer_util import generator, host_bits, normal
from test_gpu_norm import assert_same_casts

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


# rows in registers (whole and partial chunks, one and two a lane), and read twice
@pytest.mark.parametrize("K", [100, 77, 264, 1000, 1111, 8200, 16392, 16391])
@pytest.mark.parametrize("M", [5, 37, 64, 300])
def test_scales_beside_special_rows_and_weights(M, K):
    g = generator(M + K)
    x, w = normal(g, M, K), normal(g, K)
    x[0, K // 2] = NAN
    x[1, K - 1] = INF
    x[2] = 0
    x[4, :] = 1e-40
    x[M - 1, 0] = NAN
    odd = w.clone()
    odd[3], odd[K - 1], odd[K // 2] = INF, NAN, -INF
    for weight in (w, odd, None):
        for eps in (1e-6, 0.0):
            for axis in (3, 3 | mx.SCALE_TILED, 3 | mx.SCALE_TILED | mx.ELEM_E5M2 | mx.SCALE_ROUND_UP):
                o = mx.mx_rmsnorm(x.cuda(), None if weight is None else weight.cuda(), eps=eps, axis=axis,
                                  want_y=True)
                torch.cuda.synchronize()
                assert bool(o["y"][0].isnan().all()) and bool(o["y"][2].isnan().any()) == (eps == 0 or weight is odd)
                assert_same_casts(o, host_bits(o["y"]), axis)
