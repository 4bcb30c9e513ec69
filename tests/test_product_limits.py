"""The products' size limits as the header states them (no GPU): what is just inside is
planned (hostcheck stand-ins cover random sizes), what is just outside is refused before
any memory is touched.  Addresses are far apart and never read."""
import ctypes

import pytest

import block_scaled_precision_bf16_amd as mx

FAR = 1 << 44


def grouped(fn, N, K, rows):
    arr = (ctypes.c_int64 * len(rows))(*rows)
    return getattr(mx.lib(), fn)(FAR, 2 * FAR, 3 * FAR, 4 * FAR, N, K, ctypes.addressof(arr), len(rows), 0,
                                 5 * FAR, None, 0, None)


@pytest.mark.parametrize("M,N", [(1 << 23, 1 << 17), (1 << 17, 1 << 23), (1 << 20, 1 << 20)])
def test_outputs_of_the_largest_product(M, N):
    """2^40 outputs are 2^24 tiles, which a launch does not have."""
    assert mx.lib().mx_matmul(FAR, 2 * FAR, 3 * FAR, 4 * FAR, M, N, 128, 0, 5 * FAR, None, 0,
                              None) == mx.MX_ERR_SHAPE
    assert mx.mx_matmul_workspace_size(M, N, 128) == 0


@pytest.mark.parametrize("fn", ["mx_matmul_grouped", "mx_matmul_wgrad_grouped"])
def test_all_experts_weights(fn):
    """G * N * K <= 2^40, and no more than 2^23 rows in all."""
    assert grouped(fn, 1 << 20, 1 << 15, [1] * 33) == mx.MX_ERR_SHAPE
    assert grouped(fn, 64, 64, [1 << 22, (1 << 22) + 1]) == mx.MX_ERR_SHAPE
    assert grouped(fn, 64, 64, [1 << 23] * 2) == mx.MX_ERR_SHAPE
