"""The rows' gradient where slots name nothing: zeros for every number outside the slots,
as moe_gather reads them, at each row length and for rows enough to be streamed."""
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from layer_util import generator, normal

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("T,top,rows,K", [(5, 3, 40, 24), (64, 2, 300, 77), (700, 4, 5000, 7168)])
def test_rows_without_a_slot_get_zeros(T, top, rows, K):
    g = generator(rows)
    n = T * top
    slots = torch.randperm(rows, generator=g).to(I32)
    none = slots >= n                       # T * top, just past the last slot, among them
    odd = torch.tensor([-1, -2, n, n + 7, 2 ** 31 - 1, -2 ** 31], dtype=I32)
    slots[none] = torch.where(slots[none] == n, n, odd[torch.randint(0, 6, (int(none.sum()),), generator=g)])
    pos = torch.empty(n, dtype=I32)
    pos[slots[~none].long()] = torch.arange(rows, dtype=I32)[~none]
    y, dout, w = normal(g, rows, K).cuda(), normal(g, T, K).cuda(), torch.randn(T, top, generator=g).cuda()
    dy = torch.full((rows, K), 7.0, dtype=BF16, device="cuda")
    o = mx.moe_combine_backward(dout, y, w, pos=pos.view(T, top).cuda(), slots=slots.cuda(), out=dict(dy=dy))
    torch.cuda.synchronize()
    at = slots.clamp(0, n - 1).long().cuda()
    want = w.view(-1)[at, None] * dout[at // top].float()
    want[none.cuda()] = 0
    assert torch.equal(o["dy"], want.to(BF16))
