"""Gradients of a row that holds Inf (rstd 0, the Inf's xhat NaN): NaN in that row, from
bf16 and from the 8-bit copy, in each kernel; the other rows as without it, and the weight
gradients NaN only where the Inf's place, or its block in 8 bits, reaches them."""
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from layer_util import generator, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [256, 100, 8200, 16392, 16391])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_gradients_of_a_row_with_inf(K, value):
    g = generator(K)
    M, r, k = 9, 5, 70
    x, dy, w = normal(g, M, K), normal(g, M, K), normal(g, K)

    def grads(x):
        f = mx.mx_rmsnorm(x.cuda(), w.cuda(), checkpoint=True)
        return f["rstd"], [mx.mx_rmsnorm_backward(dy.cuda(), f["rstd"], w.cuda(), **src)
                           for src in (dict(h=f["h"]), dict(q_h=f["q_h"], s_h=f["s_h"]))]

    _, clean = grads(x)
    x[r, k] = value
    rstd, got = grads(x)
    assert rstd[r] == 0
    rest = [i for i in range(M) if i != r]
    for (o, c), (first, last) in zip(zip(got, clean), ((k, k + 1), (64, 96))):
        assert bool(o["dh"][r].isnan().all())
        assert torch.equal(o["dh"][rest], c["dh"][rest])
        nan = torch.zeros(K, dtype=torch.bool, device="cuda")
        nan[first:last] = True
        assert torch.equal(o["dweight"].isnan(), nan)
