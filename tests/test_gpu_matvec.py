"""NVFP4 matrix-vector products against 64-bit references: nvfp4_matvec and
nvfp4_matvec_experts.

Exact operands: codes drawn from all 16, block scales from {1/4, 1/2, 1, 3/2,
2}, tokens integers of magnitude up to 8: every product is a multiple of 1/16
(codes are multiples of 1/2, scales of 1/4; 1/2 * 3/2 needs 1/4 * 1/2) of
magnitude at most 96, so sums of up to 2^13 of them are exact in fp32 in any
order, and with a power-of-two tensor scale the output must equal the 64-bit
product rounded once.  General operands: product_util's tolerance (products of
an 8-bit and a 6-bit significand are exact in fp32) with one more half unit in
fp32, 2^-24 relative, for the tensor scale's multiplication.
"""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
import workloads as W
from product_util import E2M1, E4M3, Guarded, assert_close, assert_equal, nv_values, product, to_dev

pytestmark = pytest.mark.gpu

DT = {0: torch.bfloat16, mx.OUT_F32: torch.float32}
SCALES = np.array([int(np.argwhere(E4M3 == v)[0, 0]) for v in (0.25, 0.5, 1.0, 1.5, 2.0)], np.uint8)


def exact_weight(N, K, seed):
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, size=(N, K + K % 2)).astype(np.uint8)
    if K % 2:
        code[:, K] = 0
    return code[:, 0::2] | code[:, 1::2] << 4, SCALES[rng.integers(0, 5, size=(N, -(-K // 16)))]


def exact_tokens(T, K, seed):
    return W.bf16_bits(np.random.default_rng(seed).integers(-8, 9, size=(T, K)).astype(np.float32))


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def sg_of(*v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def values(bits):
    return W.bf16_to_f32(bits).astype(np.float64)


SHAPES = [(1, 1, 1), (1, 15, 16), (2, 16, 17), (3, 17, 32), (1, 64, 64), (5, 63, 33), (8, 100, 255),
          (15, 257, 256), (16, 48, 257), (17, 130, 512), (31, 65, 1000), (33, 16, 2048),
          (64, 96, 1024), (65, 40, 736), (130, 33, 96), (1, 1000, 4096), (4, 300, 4095),
          (16, 512, 8192), (2, 31, 7184), (1, 4096, 288), (200, 18, 48)]


@pytest.mark.parametrize("out", [0, mx.OUT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_exact(T, N, K, out):
    x = exact_tokens(T, K, T + N)
    q, s = exact_weight(N, K, N + K)
    y = Guarded((T, N), DT[out])
    r = mx.nvfp4_matvec(to_dev(x), dev(q), dev(s), sg_of(0.125), flags=out, out=y.t)
    torch.cuda.synchronize()
    assert r is y.t
    y.check("matvec")
    assert_equal(y.t, product(values(x), nv_values(q, s, 0.125, N, K))[0], f"{T} {N} {K}")


@pytest.mark.parametrize("two_d", [False, True], ids=["1d", "2d"])
@pytest.mark.parametrize("T,N,K", [(1, 512, 2048), (7, 333, 1111), (16, 256, 4096), (64, 128, 640)])
def test_quantised_weights(T, N, K, two_d):
    w = mx.nvfp4_quantize_transpose(to_dev(W.student_t_rows(N, K, 3)), axis=mx.ROWWISE, two_d=two_d)
    x = W.loguniform_rows(T, K, 4)
    v = nv_values(w["q_row"].cpu().numpy(), w["s_row"].cpu().numpy(), w["sg"].item(), N, K)
    want, mag = product(values(x), v)
    for flags in (0, mx.OUT_F32):
        y = mx.nvfp4_matvec(to_dev(x), w["q_row"], w["s_row"], w["sg"], flags=flags)
        assert_close(y, want, mag, K + 1, f"{T} {N} {K} {flags}")


def test_transposed_weights():
    """x W through the cast's transposed outputs."""
    N, K, T = 192, 272, 3
    w = mx.nvfp4_quantize_transpose(to_dev(W.normal(N, K, 5)), axis=mx.COLWISE)
    x = W.normal(T, N, 6)
    v = nv_values(w["q_col"].cpu().numpy(), w["s_col"].cpu().numpy(), w["sg"].item(), K, N)
    want, mag = product(values(x), v)
    assert_close(mx.nvfp4_matvec(to_dev(x), w["q_col"], w["s_col"], w["sg"]), want, mag, N + 1, "W^T")


@pytest.mark.parametrize("T", [1, 3, 16, 40])
def test_every_scale_code(T):
    """All 256 E4M3 scale bytes, NaN ones included, and both zeros."""
    N, K = 256, 32
    rng = np.random.default_rng(7)
    q = rng.integers(0, 256, size=(N, K // 2)).astype(np.uint8)
    s = np.stack([np.arange(256), np.full(256, 0x38)], axis=1).astype(np.uint8)
    x = exact_tokens(T, K, 8)
    v = nv_values(q, s, 1.0, N, K)
    nan = np.isnan(v).any(axis=1)
    assert nan.sum() == 2
    want, mag = product(values(x), np.nan_to_num(v))
    want[:, nan] = np.nan
    y = mx.nvfp4_matvec(to_dev(x), dev(q), dev(s), sg_of(1.0), flags=mx.OUT_F32)
    assert_close(y, want, mag, K + 1, "scale codes")


@pytest.mark.parametrize("T", [1, 6, 20])
def test_infinite_and_nan_tokens_stay_in_their_rows(T):
    N, K = 70, 300
    x = exact_tokens(T, K, 9)
    q, s = exact_weight(N, K, 10)
    q[:, 5] |= 0x11                     # no zero code where x is infinite
    v = nv_values(q, s, 1.0, N, K)
    want = product(values(x), v)[0]
    x[T - 1, 10] = 0x7F80
    want[T - 1] = np.where(v[:, 10] > 0, np.inf, -np.inf)
    if T > 1:
        x[1, 299] = 0x7FC0
        want[1] = np.nan
    y = mx.nvfp4_matvec(to_dev(x), dev(q), dev(s), sg_of(1.0))
    assert_equal(y, want, "non-finite tokens")


def test_non_finite_weights():
    """The cast of a tensor with a NaN (scale bytes 0x7F): every output NaN."""
    w = W.normal(32, 64, 1)
    w[3, 3] = 0x7FC0
    c = mx.nvfp4_quantize_transpose(to_dev(w), axis=mx.ROWWISE)
    y = mx.nvfp4_matvec(to_dev(W.normal(2, 64, 2)), c["q_row"], c["s_row"], c["sg"])
    assert bool(y.isnan().all())


def experts_want(x, e, q, s, sg, N, K):
    T, top = e.shape
    want = np.zeros((T, top, N))
    mag = np.zeros((T, top, N))
    for g in range(len(sg)):
        v = nv_values(q[g * N:(g + 1) * N], s[g * N:(g + 1) * N], sg[g], N, K)
        w, m = product(values(x), v)
        hit = e == g
        want += np.where(hit[:, :, None], w[:, None], 0)
        mag += np.where(hit[:, :, None], m[:, None], 0)
    return want, mag


CASES = [(1, 1, 1, 16, 32), (1, 2, 8, 100, 256), (1, 8, 4, 64, 512), (5, 2, 8, 33, 257),
         (16, 4, 16, 96, 320), (32, 4, 3, 48, 1024), (64, 2, 64, 40, 96), (100, 3, 5, 17, 300),
         (300, 1, 2, 31, 64), (40, 6, 1, 130, 2048), (3, 64, 7, 20, 48), (1100, 2, 9, 16, 32)]


@pytest.mark.parametrize("out", [0, mx.OUT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,top,G,N,K", CASES)
def test_experts_exact(T, top, G, N, K, out):
    rng = np.random.default_rng(T + N)
    x = exact_tokens(T, K, 1)
    q, s = exact_weight(G * N, K, 2)
    sg = [2.0 ** -(g % 5) for g in range(G)]
    # repeated experts, and slots without one: -1, G, and far values
    e = rng.integers(0, G, size=(T, top)).astype(np.int32)
    e[rng.random((T, top)) < 0.2] = rng.choice(np.array([-1, G, 2 ** 31 - 1, -2 ** 31], np.int64)
                                               ).astype(np.int32)
    y = Guarded((T, top, N), DT[out])
    mx.nvfp4_matvec_experts(to_dev(x), dev(e), dev(q), dev(s), sg_of(*sg), flags=out, out=y.t)
    torch.cuda.synchronize()
    y.check("experts")
    assert_equal(y.t, experts_want(x, e, q, s, sg, N, K)[0], f"{T} {top} {G}")


def test_experts_of_one_choice_and_of_none():
    T, top, G, N, K = 20, 2, 4, 50, 200
    x = exact_tokens(T, K, 1)
    q, s = exact_weight(G * N, K, 2)
    sg = [1.0] * G
    for e in (np.full((T, top), 2, np.int32), np.full((T, top), -1, np.int32)):
        y = mx.nvfp4_matvec_experts(to_dev(x), dev(e), dev(q), dev(s), sg_of(*sg))
        assert_equal(y, experts_want(x, e, q, s, sg, N, K)[0], str(e[0, 0]))


def test_nan_expert_touches_its_slots_only():
    T, top, G, N, K = 9, 2, 3, 32, 64
    x = exact_tokens(T, K, 1)
    q, s = exact_weight(G * N, K, 2)
    e = np.random.default_rng(3).integers(0, G, size=(T, top)).astype(np.int32)
    want = experts_want(x, e, q, s, [1.0] * G, N, K)[0]
    want[e == 1] = np.nan
    s[N:2 * N] = 0x7F
    y = mx.nvfp4_matvec_experts(to_dev(x), dev(e), dev(q), dev(s), sg_of(1.0, 1.0, 1.0))
    assert_equal(y, want, "NaN expert")


def test_experts_quantised_by_the_grouped_cast_and_both_projections():
    """Decoding through an MoE layer: up projection per slot, SwiGLU, and the
    down projection of the slots' own rows (top = 1)."""
    T, top, G, D, H = 6, 2, 4, 160, 96
    w1 = to_dev(W.normal(G * 2 * H, D, 1, 0.1))
    w2 = to_dev(W.normal(G * D, H, 2, 0.1))
    r1, r2 = [2 * H] * G, [D] * G
    c1 = mx.nvfp4_quantize_transpose_grouped(w1, r1, mx.mx_absmax_bf16_grouped(w1, r1), axis=mx.ROWWISE)
    c2 = mx.nvfp4_quantize_transpose_grouped(w2, r2, mx.mx_absmax_bf16_grouped(w2, r2), axis=mx.ROWWISE)
    x = W.normal(T, D, 3)
    e = np.random.default_rng(4).integers(-1, G, size=(T, top)).astype(np.int32)
    h = mx.nvfp4_matvec_experts(to_dev(x), dev(e), c1["q_row"], c1["s_row"], c1["sg"])
    want, mag = experts_want(x, e, c1["q_row"].cpu().numpy(), c1["s_row"].cpu().numpy(),
                             c1["sg"].tolist(), 2 * H, D)
    assert_close(h, want, mag, D + 1, "up")
    a = mx.mx_fused_values(h.view(T * top, 2 * H).view(torch.int16), op=mx.OP_GATED | mx.GATED_SWIGLU)
    e2 = e.reshape(-1, 1)
    y = mx.nvfp4_matvec_experts(a, dev(e2), c2["q_row"], c2["s_row"], c2["sg"], flags=mx.OUT_F32)
    ab = a.cpu().numpy().view(np.uint16)
    want, mag = experts_want(ab, e2, c2["q_row"].cpu().numpy(), c2["s_row"].cpu().numpy(),
                             c2["sg"].tolist(), D, H)
    assert_close(y, want, mag, H + 1, "down")


def test_captured_on_another_stream_and_repeats():
    T, top, G, N, K = 8, 2, 4, 200, 512
    q, s = exact_weight(G * N, K, 2)
    q, s, sg = dev(q), dev(s), sg_of(*[1.0] * G)
    xs = [to_dev(W.normal(T, K, i)) for i in (1, 2, 3)]
    es = [dev(np.random.default_rng(i).integers(-1, G + 1, size=(T, top)).astype(np.int32))
          for i in (1, 2, 3)]
    x, e = xs[0].clone(), es[0].clone()

    def step():
        return (mx.nvfp4_matvec_experts(x, e, q, s, sg),
                mx.nvfp4_matvec(x, q[:N], s[:N], sg[:1]))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = step()
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        e.copy_(es[i])
        graph.replay()
        torch.cuda.synchronize()
        got = a.clone(), b.clone()
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = mx.nvfp4_matvec_experts(x, e, q, s, sg, stream=st)
    st.synchronize()
    assert torch.equal(other, step()[0])


@pytest.mark.parametrize("T,N,K,G", [
    (1, 65600, 131088, 0), (20, 65600, 131088, 0),       # codes past 2^32 bytes
    (32800, 32800, 32, 0), (70001, 64, 32784, 0),        # the output, the tokens
    (3, 16400, 8208, 66), (100, 16400, 8208, 66)])       # the last experts' codes
def test_past_32_bits(T, N, K, G):
    """Exact operands made on the GPU: tokens n in {-4 .. 4}, scales 1/2, 1 and 2,
    so products are multiples of 1/4 and no sum here passes 2^24 of them."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    rows = max(G, 1) * N

    def bytes_(r, c, lo=0, hi=256):
        return torch.randint(lo, hi, (r, c), dtype=torch.uint8, device="cuda", generator=gen)

    qw, sw, x = bytes_(rows, K // 2), 0x30 + 8 * bytes_(rows, K // 16, 0, 3), torch.empty(
        T, K, dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 8192):
        x[i:i + 8192] = bytes_(min(8192, T - i), K, 0, 9) - 4.0
    e2m1 = torch.from_numpy(E2M1).cuda()

    def weights(r):
        q = qw[r].int()
        v = e2m1[torch.stack([q & 15, q >> 4], dim=-1).view(len(r), K)]
        return v * torch.exp2((sw[r].double() - 0x38) / 8).repeat_interleave(16, 1)

    cpu = torch.Generator().manual_seed(6)
    n = torch.cat([torch.tensor([0, N - 1]), torch.randint(0, N, (20,), generator=cpu)]).cuda()
    t = torch.cat([torch.tensor([0, T - 1]), torch.randint(0, T, (6,), generator=cpu)]).cuda()
    sg = torch.ones(max(G, 1), device="cuda")
    if not G:
        y = mx.nvfp4_matvec(x, qw, sw, sg, flags=mx.OUT_F32)
        assert torch.equal(y[t][:, n].double(), x[t].double() @ weights(n).t())
        return
    e = torch.randint(G - 3, G, (T, 2), dtype=torch.int32, device="cuda", generator=gen)
    y = mx.nvfp4_matvec_experts(x, e, qw, sw, sg, flags=mx.OUT_F32)
    for i in t.tolist():
        for j in range(2):
            w = weights(int(e[i, j]) * N + n)
            assert torch.equal(y[i, j, n].double(), w @ x[i].double())
