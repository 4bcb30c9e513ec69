"""Weight gradients added to an existing tensor: an empty expert's part is left as it
was, to the bit (-0 and the payloads of NaNs too), by each kernel."""
import pytest
import torch

import block_scaled_precision_bf16_amd as mx

pytestmark = pytest.mark.gpu


# below one load, small, 128 x 128 tiles, 256 x 256 tiles, copied rows
@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("rows,N,K", [([0, 1, 0], 5, 7), ([64, 0, 33], 96, 160), ([512, 0, 512], 1024, 2048),
                                      ([4096, 0, 2048], 2048, 2304), ([2049, 0, 1000], 2048, 2304)])
def test_empty_groups_keep_their_bits(rows, N, K, tiled):
    gen = torch.Generator(device="cuda").manual_seed(1)
    bits = torch.randint(-2 ** 31, 2 ** 31, (len(rows), N, K), device="cuda", generator=gen).to(torch.int32)
    bits[0] = -2 ** 31                             # -0
    for g, r in enumerate(rows):
        if r == 0:
            bits[g, 0, :3] = torch.tensor([-2 ** 31, 0x7FA00001, -0x3FFFFF], dtype=torch.int32)
    y = bits.clone().view(torch.float32)
    codes = [torch.full((n * sum(rows),), 0x38, dtype=torch.uint8, device="cuda") for n in (N, K)]

    def scales(n):
        def size(r):
            return -(-n // 32) * -(-r // 256) * 256 if tiled else n * -(-r // 32)
        return torch.full((sum(size(r) for r in rows),), 127, dtype=torch.uint8, device="cuda")

    mx.mx_matmul_wgrad_grouped(codes[0], scales(N), codes[1], scales(K), rows,
                               flags=tiled | mx.OUT_F32 | mx.ACCUMULATE, out=y)
    for g, r in enumerate(rows):
        if r == 0:
            assert torch.equal(y[g].view(torch.int32), bits[g]), f"group {g}"
    full = [g for g, r in enumerate(rows) if r][0]
    if full == 0:
        assert bool((y[0] == rows[0]).all())       # -0 + sum of ones
