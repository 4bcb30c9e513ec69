"""MXFP8 products over the whole range of scale bytes and at the border of what the
8-bit matrix instruction keeps, by each kernel.

One operand is dense, the other holds one or two elements a row, so that an
output is one product, or the sum of two, and is known exactly without a matrix
product:
  - one element, bytes of both operands from both ends and the middle of 0 .. 254:
    the product (at most 8 significant bits) has to be right to the bit.  Below
    2^-126 it is a multiple of 2^-149 after one rounding, off by half of that;
    adding zeros to it and rounding it to bf16 (there a multiple of 2^-133) are
    exact, or one more half step;
  - two elements among 8 neighbouring k, whose products are up to 2^16 apart (17
    bits of sum): fp32 outputs have to be right to the bit, which sums that drop
    what is below 2^-13 of the larger one (bf16 outputs) are not.
"""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from product_cases import PRODUCTS
from product_util import E4M3, E5M2
from test_gpu_matmul_tiles import tiled_layout

pytestmark = pytest.mark.gpu

ENDS = [*range(0, 13), *range(117, 138), *range(236, 255)]
SIZES = [size for size, _ in PRODUCTS]       # each kernel


def finite_codes(e5m2):
    t = E5M2 if e5m2 else E4M3
    return np.flatnonzero(np.isfinite(t)).astype(np.uint8)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def values(codes, e5m2):
    return dev(E5M2 if e5m2 else E4M3)[codes.int()]


def scale_of(byte):
    return torch.where(byte == 255, float("nan"), torch.exp2(byte.double() - 127))


def operand(s, tiled):
    return tiled_layout(s) if tiled else s.view(-1)


def assert_product(got, want, what):
    """got: the exact values `want` after one rounding to fp32 and, for bf16 outputs,
    another to bf16."""
    f = want.float().to(got.dtype).double()
    g = got.double()
    step = 2.0 ** -149 if got.dtype == torch.float32 else 2.0 ** -133
    ok = (g == f) | (g.isnan() & want.isnan()) | ((want.abs() < 2.0 ** -126) & ((g - want).abs() <= step))
    if not bool(ok.all()):
        bad = (~ok).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {len(bad)} of {ok.numel()} wrong, first at {i}: "
                             f"{got[i].item()} for {want[i].item()}")


def multiply(dense, one, dense_is_a, M, N, K, flags):
    (qd, sd), (qo, so) = dense, one
    a, b = ((qd, sd), (qo, so)) if dense_is_a else ((qo, so), (qd, sd))
    y = mx.mx_matmul(a[0], operand(a[1], flags & mx.SCALE_TILED), b[0],
                     operand(b[1], flags & mx.SCALE_TILED), flags=flags)
    return y if dense_is_a else y.t()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "mixed"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_every_scale_byte(M, N, K, fmt):
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    for dense_is_a in (True, False):
        R, C = (M, N) if dense_is_a else (N, M)
        ed, eo = fmt != "e4m3", fmt == "e5m2"
        nb = -(-K // 32)

        def pick(table, *shape):
            t = dev(np.asarray(table, np.uint8))
            return t[torch.randint(0, len(t), shape, device="cuda", generator=gen)]

        qd, sd = pick(finite_codes(ed), R, K), pick(ENDS, R, nb)
        at = torch.randint(0, K, (C,), device="cuda", generator=gen)
        co, so = pick(finite_codes(eo), C), pick(ENDS, C, nb)
        qo = torch.zeros(C, K, dtype=torch.uint8, device="cuda")
        cols = torch.arange(C, device="cuda")
        qo[cols, at] = co
        want = values(qd[:, at], ed) * scale_of(sd[:, at // 32]) * \
            (values(co, eo) * scale_of(so[cols, at // 32]))
        fl = (mx.A_E5M2 if (ed if dense_is_a else eo) else 0) | (mx.B_E5M2 if (eo if dense_is_a else ed) else 0)
        for flags in (0, mx.SCALE_TILED, mx.OUT_F32, mx.OUT_F32 | mx.SCALE_TILED):
            y = multiply((qd, sd), (qo, so), dense_is_a, M, N, K, fl | flags)
            assert_product(y, want, f"{M}x{N}x{K} {fmt} {dense_is_a} {flags}")


def test_nan_blocks_among_far_ones():
    M, N, K = 300, 200, 400
    gen = torch.Generator(device="cuda").manual_seed(1)
    qd = torch.randint(0, 127, (M, K), dtype=torch.uint8, device="cuda", generator=gen)
    sd = torch.randint(0, 255, (M, 13), dtype=torch.uint8, device="cuda", generator=gen)
    qd[7, 64:96], sd[7, 2] = 0x7F, 255
    at = torch.randint(0, K, (N,), device="cuda", generator=gen)
    qo = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    so = torch.randint(0, 255, (N, 13), dtype=torch.uint8, device="cuda", generator=gen)
    cols = torch.arange(N, device="cuda")
    qo[cols, at] = 0x38
    want = values(qd[:, at], False) * scale_of(sd[:, at // 32]) * scale_of(so[cols, at // 32])
    want[7] = float("nan")
    for flags in (0, mx.SCALE_TILED, mx.OUT_F32, mx.OUT_F32 | mx.SCALE_TILED):
        assert_product(multiply((qd, sd), (qo, so), True, M, N, K, flags), want, str(flags))


def test_largest_values_of_the_round_up_cast():
    """bf16's largest number rounds up to 2^128 in a block of its own scale: finite
    products with small operands."""
    K = 64
    x = np.full((40, K), 0x7F7F, np.uint16)
    w = np.full((48, K), 0x0C00 | 0x0080, np.uint16)                # 2^-102
    for e5 in (0, mx.ELEM_E5M2):
        c = mx.mx_quantize(dev(x.view(np.int16)), axis=mx.ROWWISE | mx.SCALE_ROUND_UP | e5)
        d = mx.mx_quantize(dev(w.view(np.int16)), axis=mx.ROWWISE | mx.SCALE_ROUND_UP)
        a = values(c["q_row"], bool(e5)) * scale_of(c["s_row"]).repeat_interleave(32, 1)
        b = values(d["q_row"], False) * scale_of(d["s_row"]).repeat_interleave(32, 1)
        assert bool((a == 2.0 ** 128).all())
        for flags in (0, mx.OUT_F32):
            y = mx.mx_matmul(c["q_row"], c["s_row"], d["q_row"], d["s_row"],
                             flags=flags | (mx.A_E5M2 if e5 else 0))
            assert_product(y, a @ b.t(), f"{e5} {flags}")


@pytest.mark.parametrize("far", [False, True], ids=["near", "far"])
@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_fp32_outputs_drop_nothing(M, N, K, tiled, far):
    """Sums of +-2^8 and +-2^-8 (or of two of one size) among 8 neighbouring k."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    nb = -(-K // 32)
    codes = dev(np.array([int(np.flatnonzero(E4M3 == v)[0]) for v in (16., -16., 2. ** -4, -2. ** -4)],
                         np.uint8))
    qd = codes[torch.randint(0, 4, (M, K), device="cuda", generator=gen)]
    k1 = torch.randint(0, K, (N,), device="cuda", generator=gen)
    k2 = k1 // 8 * 8 + (k1 % 8 + torch.randint(1, 8, (N,), device="cuda", generator=gen)) % 8
    k2 = torch.where(k2 < K, k2, k1 // 8 * 8)
    cols = torch.arange(N, device="cuda")
    qo = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    qo[cols, k1], qo[cols, k2] = codes[0], codes[2]
    up = 121 if far else 0            # bytes 248 and 6: the dense operand's blocks are far
    sd = torch.full((M, nb), 127 + up, dtype=torch.uint8, device="cuda")
    so = torch.full((N, nb), 127 - up, dtype=torch.uint8, device="cuda")
    vo = values(qo, False)
    want = values(qd[:, k1], False) * vo[cols, k1] + \
        torch.where(k1 == k2, 0.0, values(qd[:, k2], False) * vo[cols, k2])
    flags = tiled | mx.OUT_F32
    assert_product(multiply((qd, sd), (qo, so), True, M, N, K, flags), want, f"{M}x{N}x{K}")


def test_grouped_products_and_weight_gradients_of_far_blocks():
    rows, N, K = [70, 0, 33, 129], 160, 224
    G, M = len(rows), sum(rows)
    gen = torch.Generator(device="cuda").manual_seed(5)
    ends = dev(np.asarray(ENDS, np.uint8))

    def pick(*shape):
        return ends[torch.randint(0, len(ends), shape, device="cuda", generator=gen)]

    def one(n, k):
        """[n][k] with an element 1 in each row."""
        q = torch.zeros(n, k, dtype=torch.uint8, device="cuda")
        at = torch.randint(0, k, (n,), device="cuda", generator=gen)
        q[torch.arange(n, device="cuda"), at] = 0x38
        return q, pick(n, -(-k // 32)), at

    def want(q, s, o):
        n = torch.arange(len(o[2]), device="cuda")
        return values(q[:, o[2]], False) * scale_of(s[:, o[2] // 32]) * scale_of(o[1][n, o[2] // 32])

    qa, sa = torch.randint(0, 127, (M, K), dtype=torch.uint8, device="cuda", generator=gen), pick(M, K // 32)
    bs = [one(N, K) for _ in rows]
    y = mx.mx_matmul_grouped(qa, sa.view(-1), torch.cat([b[0] for b in bs]),
                             torch.cat([b[1].view(-1) for b in bs]), rows, flags=mx.OUT_F32)
    parts = torch.split(qa, rows), torch.split(sa, rows)
    assert_product(y, torch.cat([want(q, s, b) for q, s, b in zip(*parts, bs)]), "by expert")

    ds = [(torch.randint(0, 127, (N, r), dtype=torch.uint8, device="cuda", generator=gen), pick(N, -(-r // 32)))
          for r in rows]
    xs = [one(K, r) if r else None for r in rows]
    dw = mx.mx_matmul_wgrad_grouped(torch.cat([q.view(-1) for q, _ in ds]), torch.cat([s.view(-1) for _, s in ds]),
                                    torch.cat([x[0].view(-1) for x in xs if x]),
                                    torch.cat([x[1].view(-1) for x in xs if x]), rows, flags=mx.OUT_F32)
    for g, r in enumerate(rows):
        w = want(*ds[g], xs[g]) if r else torch.zeros(N, K, dtype=torch.float64, device="cuda")
        assert_product(dw[g], w, f"weight gradient {g}")


@pytest.mark.parametrize("far", [False, True], ids=["near", "far"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_infinite_and_nan_elements(M, N, K, far):
    """E5M2 has infinities, and both formats NaNs, which the casts do not write but an
    operand may hold: +-Inf times a number, NaN times anything, in the rows that hold
    them only."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    nb = -(-K // 32)
    qa = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    qb = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    at = K // 2
    qb[:, at] = 0x38 | (torch.randint(0, 2, (N,), device="cuda", generator=gen) * 0x80).byte()   # +-1
    qa[:, at] = 0x3C                                                  # E5M2 1
    kinds = dev(np.array([0x3C, 0x7C, 0xFC, 0x7D, 0xFF], np.uint8))   # 1, Inf, -Inf, NaN, NaN
    which = torch.randint(0, 5, (M,), device="cuda", generator=gen)
    which[-1] = 1
    qa[:, at] = kinds[which]
    up = 121 if far else 0
    sa = torch.full((M, nb), 127 + up, dtype=torch.uint8, device="cuda")
    sb = torch.full((N, nb), 127 - up, dtype=torch.uint8, device="cuda")
    a = dev(np.array([1, np.inf, -np.inf, np.nan, np.nan]))[which]
    want = a[:, None] * values(qb[:, at], False)[None]
    for flags in (0, mx.SCALE_TILED, mx.OUT_F32, mx.OUT_F32 | mx.SCALE_TILED):
        y = multiply((qa, sa), (qb, sb), True, M, N, K, flags | mx.A_E5M2)
        assert_product(y, want, f"{M}x{N}x{K} {flags}")
    qa[:, at] = 0x38
    qa[0, at] = 0x7F                                                  # E4M3 NaN
    want = torch.ones(M, 1, dtype=torch.float64, device="cuda") * values(qb[:, at], False)[None]
    want[0] = float("nan")
    for flags in (0, mx.SCALE_TILED, mx.OUT_F32, mx.OUT_F32 | mx.SCALE_TILED):
        y = multiply((qa, sa), (qb, sb), True, M, N, K, flags)
        assert_product(y, want, f"{M}x{N}x{K} {flags} E4M3")


@pytest.mark.parametrize("M,N,K", SIZES)
def test_nan_blocks_of_zeros(M, N, K):
    """A block's scale alone makes it NaN, whatever its elements."""
    nb = -(-K // 32)
    for e5m2 in (False, True):
        q = torch.full((M, K), 0x3C if e5m2 else 0x38, dtype=torch.uint8, device="cuda")
        s = torch.full((M, nb), 127, dtype=torch.uint8, device="cuda")
        qo = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
        qo[:, 0] = 0x38
        so = torch.full((N, nb), 127, dtype=torch.uint8, device="cuda")
        q[M - 1, 32 * (nb - 1):], s[M - 1, nb - 1] = 0, 255
        so[0, nb // 2], qo[0, 32 * (nb // 2):32 * (nb // 2) + 32] = 255, 0
        want = torch.ones(M, N, dtype=torch.float64, device="cuda")
        want[M - 1], want[:, 0] = float("nan"), float("nan")
        for flags in (0, mx.SCALE_TILED, mx.OUT_F32, mx.OUT_F32 | mx.SCALE_TILED):
            y = multiply((q, s), (qo, so), True, M, N, K, flags | (mx.A_E5M2 if e5m2 else 0))
            assert_product(y, want, f"{M}x{N}x{K} {e5m2} {flags}")
