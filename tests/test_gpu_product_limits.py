"""Products with sums of 2^23, the longest, so that a tile's last row lies about 2^31
bytes behind its first and the kernels' 32-bit offsets run up to the largest buffer
descriptor.

The operands are zero but for planted columns (both ends and some between), the same
in all rows, with exact elements (product_util's kind, made as codes), so that an
output must equal the 64-bit product of those columns rounded once: at most 448
products that are multiples of 1/4 and 64 at most, below 2^24 quarters.
"""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from product_util import E2M1, E4M3
from test_gpu_matmul_tiles import DT, assert_same, codes_of, tiled_layout

pytestmark = pytest.mark.gpu

LONG = 1 << 23


def planted(K, gen):
    ends = torch.arange(64, device="cuda")
    some = torch.randint(64, K - 64, (320,), device="cuda", generator=gen)
    return torch.cat([ends, some, K - 1 - ends]).unique()


def operand(rows, K, cols, gen):
    """Codes, scale bytes and the planted columns' values."""
    n = torch.randint(0, 9, (rows, len(cols)), device="cuda", generator=gen)
    s = torch.randint(126, 129, (rows, -(-K // 32)), dtype=torch.uint8, device="cuda", generator=gen)
    q = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
    q[:, cols] = torch.from_numpy(codes_of(E4M3)).cuda()[n]
    return q, s, (n - 4).double() * torch.exp2(s[:, cols // 32].double() - 127)


# the small products' kernel, aligned and not, and the tiled one's parts
@pytest.mark.parametrize("M,N,K", [(130, 70, LONG), (33, 100, LONG - 7), (256, 4096, LONG), (250, 4095, LONG - 16)])
def test_longest_sums(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(1)
    cols = planted(K, gen)
    qa, sa, va = operand(M, K, cols, gen)
    qb, sb, vb = operand(N, K, cols, gen)
    want = va @ vb.t()
    for flags in (0, mx.SCALE_TILED, mx.OUT_F32, mx.OUT_F32 | mx.SCALE_TILED):
        lay = tiled_layout if flags & mx.SCALE_TILED else lambda s: s.view(-1)
        y = mx.mx_matmul(qa, lay(sa), qb, lay(sb), flags=flags)
        assert y.dtype == DT[flags & mx.OUT_F32]
        assert_same(y, want, f"{M}x{N}x{K} {flags}")


@pytest.mark.parametrize("T,N,K", [(1, 70, LONG), (2, 65, LONG - 1), (16, 40, LONG), (3, 70, LONG - 9)])
def test_longest_matvec(T, N, K):
    """Weights random throughout, tokens zero but for the planted columns; scales 1/2 and
    1, codes up to 6, tokens integers up to 4: multiples of 1/4 of 24 at most."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    cols = planted(K, gen)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[:, cols] = torch.randint(-4, 5, (T, len(cols)), device="cuda", generator=gen).to(torch.bfloat16)
    q = torch.randint(0, 256, (N, -(-K // 2)), dtype=torch.uint8, device="cuda", generator=gen)
    if K % 2:
        q[:, -1] &= 15
    s = 0x30 + 8 * torch.randint(0, 2, (N, -(-K // 16)), dtype=torch.uint8, device="cuda", generator=gen)
    code = (q[:, cols // 2].int() >> (4 * (cols % 2)).int()) & 15
    v = torch.from_numpy(E2M1).cuda()[code] * torch.exp2((s[:, cols // 16].double() - 0x38) / 8)
    want = x[:, cols].double() @ v.t()
    sg = torch.ones(3, device="cuda")
    assert_same(mx.nvfp4_matvec(x, q, s, sg[:1], flags=mx.OUT_F32), want, f"{T} {N} {K}")
    e = torch.full((T, 1), 2, dtype=torch.int32, device="cuda")
    y = mx.nvfp4_matvec_experts(x, e, q.repeat(3, 1), s.repeat(3, 1), sg)
    assert_same(y.view(T, N), want, f"experts {T} {N} {K}")
