"""Weight gradients of rows longer than 16384 over many of them: a bound that does not
grow with their number, at terms of one sign and size, whose roundings add up."""
import pytest
import torch

import block_scaled_precision_bf16_amd as mx

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = 2.0 ** -24


@pytest.mark.parametrize("K", [16392, 16391])
@pytest.mark.parametrize("ckpt", [False, True], ids=["bf16", "8bit"])
def test_weight_gradient_over_many_long_rows(K, ckpt):
    M = 65536
    g = torch.Generator("cuda").manual_seed(K)
    dy = (1 + torch.rand(1, K, generator=g, device="cuda")).to(BF16)
    rstd = 0.5 + torch.rand(1, generator=g, device="cuda")
    if ckpt:
        src = dict(q_h=torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda"),          # 1
                   s_h=torch.full((M, -(-K // 32)), 127, dtype=torch.uint8, device="cuda"))
    else:
        src = dict(h=torch.ones(M, K, dtype=BF16, device="cuda"))
    o = mx.mx_rmsnorm_backward(dy.expand(M, K).contiguous(), rstd.expand(M).contiguous(), **src)
    want = M * dy[0].to(F64) * rstd.to(F64)
    # h rstd is exact; 64 rows in a line (the products inside the FMA), their sums in 64
    # bits, rounded once; the 64 slices by 32 threads, and these by one
    off = ((o["dweight"].to(F64) - want).abs() / want).max().item() / HALF
    assert off <= 64 + 1 + 2 + 32, off
