"""MXFP8 products against 64-bit references: mx_matmul, mx_matmul_grouped and
mx_matmul_wgrad_grouped (operands, references and tolerances: product_util)."""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
import workloads as W
from product_util import (Guarded, assert_close, assert_equal, exact_bits, mx_values, product,
                          to_dev)

pytestmark = pytest.mark.gpu

DT = {0: torch.bfloat16, mx.OUT_F32: torch.float32}
FORMATS = [(False, False), (True, False), (False, True), (True, True)]


def fmt_flags(ea, eb):
    return (mx.A_E5M2 if ea else 0) | (mx.B_E5M2 if eb else 0)


def cast_rows(bits, flags, e5m2):
    g = mx.mx_quantize(to_dev(bits), axis=mx.ROWWISE | (flags & mx.SCALE_TILED) |
                       (mx.ELEM_E5M2 if e5m2 else 0))
    return g["q_row"], g["s_row"]


def dense(M, N, K, flags, ea, eb, seed, bits=exact_bits):
    a, b = bits(M, K, seed), bits(N, K, seed + 1)
    qa, sa = cast_rows(a, flags, ea)
    qb, sb = cast_rows(b, flags, eb)
    return qa, sa, qb, sb, mx_values(qa, sa, M, K, flags, ea), mx_values(qb, sb, N, K, flags, eb)


SHAPES = [(1, 1, 1), (1, 1, 32), (1, 7, 33), (3, 5, 16), (33, 65, 31), (64, 64, 64), (16, 128, 96),
          (128, 128, 128), (256, 256, 256), (257, 255, 130), (255, 257, 272), (100, 300, 1000),
          (31, 513, 4112), (512, 768, 2048), (300, 200, 144), (129, 127, 255), (1, 1000, 777),
          (700, 1, 640), (40, 640, 1024), (17, 96, 8192), (513, 511, 1153), (260, 520, 416)]


@pytest.mark.parametrize("out", [0, mx.OUT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_products(M, N, K, tiled, out):
    flags = tiled | out
    qa, sa, qb, sb, a, b = dense(M, N, K, flags, False, False, seed=M + 3 * N + 7 * K)
    y = Guarded((M, N), DT[out])
    r = mx.mx_matmul(qa, sa, qb, sb, flags=flags, out=y.t)
    torch.cuda.synchronize()
    assert r is y.t
    y.check("mx_matmul")
    assert_equal(y.t, product(a, b)[0], f"{M}x{N}x{K}")


@pytest.mark.parametrize("ea,eb", FORMATS)
@pytest.mark.parametrize("M,N,K", [(96, 160, 200), (256, 256, 512), (20, 300, 1000)])
def test_exact_products_of_every_format(M, N, K, ea, eb):
    for flags in (0, mx.SCALE_TILED | mx.OUT_F32):
        flags |= fmt_flags(ea, eb)
        qa, sa, qb, sb, a, b = dense(M, N, K, flags, ea, eb, seed=11)
        assert_equal(mx.mx_matmul(qa, sa, qb, sb, flags=flags), product(a, b)[0], f"{ea} {eb} {flags}")


@pytest.mark.parametrize("M,N,K", [(200, 333, 1111), (512, 512, 4096), (8, 1024, 2048),
                                   (1024, 256, 7168)])
@pytest.mark.parametrize("ea,eb", FORMATS)
def test_general_products(M, N, K, ea, eb):
    for flags in (mx.OUT_F32, mx.SCALE_TILED):
        f = flags | fmt_flags(ea, eb)
        qa, sa, qb, sb, a, b = dense(M, N, K, f, ea, eb, seed=21, bits=W.loguniform_rows)
        want, mag = product(a, b)
        assert_close(mx.mx_matmul(qa, sa, qb, sb, flags=f), want, mag, K, f"{M}x{N}x{K} {f}",
                     cut=not f & mx.OUT_F32)


@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("M,N,K", [(70, 90, 300), (256, 512, 1024), (12, 256, 640)])
def test_nan_blocks_reach_their_rows_and_columns_only(M, N, K, tiled):
    a, b = exact_bits(M, K, 5), exact_bits(N, K, 6)
    a[M // 2, K - 1] = 0x7FC0          # NaN in the last, partial block
    a[0, 3] = 0x7F80                   # Inf: a NaN block as well
    b[N - 1, 40] = 0xFFC0
    qa, sa = cast_rows(a, tiled, False)
    qb, sb = cast_rows(b, tiled, False)
    va, vb = mx_values(qa, sa, M, K, tiled), mx_values(qb, sb, N, K, tiled)
    want = product(np.nan_to_num(va), np.nan_to_num(vb))[0]
    want[M // 2], want[0], want[:, N - 1] = np.nan, np.nan, np.nan
    for flags in (tiled, tiled | mx.OUT_F32):
        assert_equal(mx.mx_matmul(qa, sa, qb, sb, flags=flags), want, "NaN blocks")


def test_extreme_scales():
    """Blocks of tiny and huge values: scale bytes near both ends."""
    M, N, K = 64, 64, 256
    rng = np.random.default_rng(3)
    e = rng.integers(-60, 60, size=(M, 1)).astype(np.float32)
    a = W.bf16_bits((rng.integers(1, 5, size=(M, K)) * np.exp2(e)).astype(np.float32))
    b = W.bf16_bits((rng.integers(1, 5, size=(N, K)) * np.exp2(-e[::-1])).astype(np.float32))
    qa, sa = cast_rows(a, 0, False)
    qb, sb = cast_rows(b, 0, False)
    want, mag = product(mx_values(qa, sa, M, K), mx_values(qb, sb, N, K))
    assert_close(mx.mx_matmul(qa, sa, qb, sb, flags=mx.OUT_F32), want, mag, K, "scales")


def test_accumulate():
    M, N, K = 130, 70, 333
    flags = mx.OUT_F32 | mx.ACCUMULATE
    qa, sa, qb, sb, a, b = dense(M, N, K, 0, False, False, seed=31)
    start = torch.randint(-100, 100, (M, N), device="cuda").float()
    y = start.clone()
    mx.mx_matmul(qa, sa, qb, sb, flags=flags, out=y)
    mx.mx_matmul(qa, sa, qb, sb, flags=flags, out=y)
    assert_equal(y, start.cpu().double().numpy() + 2 * product(a, b)[0], "accumulate")


ROWS = [[5, 0, 64, 1, 130], [64], [0, 0, 7], [32, 32, 32, 32], [1] * 20, [300, 20, 0, 0, 700],
        [256, 512, 0, 256], [16, 48, 80, 112], [3, 2, 9, 0, 11, 4, 1, 2], [0] * 63 + [40]]


def grouped(rows, N, K, flags, ea, eb, seed, bits=exact_bits):
    M, G = sum(rows), len(rows)
    tile = flags & mx.SCALE_TILED
    ga = mx.mx_quantize_grouped(to_dev(bits(M, K, seed)), rows,
                                axis=mx.ROWWISE | tile | (mx.ELEM_E5M2 if ea else 0))
    gb = mx.mx_quantize_grouped(to_dev(bits(G * N, K, seed + 1)), [N] * G,
                                axis=mx.ROWWISE | tile | (mx.ELEM_E5M2 if eb else 0))
    return ga["q_row"], ga["s_row"], gb["q_row"], gb["s_row"]


def split(q, s, shapes, flags, e5m2):
    """float64 values of operands standing one after the other."""
    q, s, out = q.view(-1), s.view(-1), []
    for r, c in shapes:
        if r == 0 or c == 0:
            out.append(np.zeros((r, c)))
            continue
        n = mx.mx_scale_size(r, c, 1 | (flags & mx.SCALE_TILED))
        out.append(mx_values(q[:r * c], s[:n], r, c, flags, e5m2))
        q, s = q[r * c:], s[n:]
    return out


@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("N,K", [(96, 160), (256, 512), (130, 77), (512, 1040)])
@pytest.mark.parametrize("rows", ROWS, ids=[str(i) for i in range(len(ROWS))])
def test_grouped_products(rows, N, K, tiled):
    M = sum(rows)
    for flags in (tiled, tiled | mx.OUT_F32 | mx.A_E5M2):
        ea = bool(flags & mx.A_E5M2)
        qa, sa, qb, sb = grouped(rows, N, K, flags, ea, False, seed=41)
        y = Guarded((M, N), DT[flags & mx.OUT_F32])
        mx.mx_matmul_grouped(qa, sa, qb, sb, rows, flags=flags, out=y.t)
        torch.cuda.synchronize()
        y.check("grouped")
        va = split(qa, sa, [(r, K) for r in rows], flags, ea)
        vb = split(qb, sb, [(N, K) for _ in rows], flags, False)
        want = np.concatenate([product(a, b)[0] for a, b in zip(va, vb)])
        assert_equal(y.t, want, f"rows {rows}")


@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("N,K", [(96, 160), (256, 512), (130, 77), (272, 300)])
@pytest.mark.parametrize("rows", ROWS, ids=[str(i) for i in range(len(ROWS))])
def test_grouped_weight_gradients(rows, N, K, tiled):
    M, G = sum(rows), len(rows)
    for flags in (tiled, tiled | mx.OUT_F32 | mx.A_E5M2):
        ea = bool(flags & mx.A_E5M2)
        # exact along the summed rows: blocks run down the columns
        dy = np.concatenate([exact_bits(N, r, 50 + i).T if r else np.zeros((0, N), np.uint16)
                             for i, r in enumerate(rows)])
        x = np.concatenate([exact_bits(K, r, 90 + i).T if r else np.zeros((0, K), np.uint16)
                            for i, r in enumerate(rows)])
        ga = mx.mx_quantize_grouped(to_dev(dy), rows,
                                    axis=mx.COLWISE | tiled | (mx.ELEM_E5M2 if ea else 0))
        gb = mx.mx_quantize_grouped(to_dev(x), rows, axis=mx.COLWISE | tiled)
        y = Guarded((G, N, K), DT[flags & mx.OUT_F32])
        mx.mx_matmul_wgrad_grouped(ga["q_col"], ga["s_col"], gb["q_col"], gb["s_col"], rows,
                                   flags=flags, out=y.t)
        torch.cuda.synchronize()
        y.check("wgrad")
        va = split(ga["q_col"], ga["s_col"], [(N, r) for r in rows], flags, ea)
        vb = split(gb["q_col"], gb["s_col"], [(K, r) for r in rows], flags, False)
        want = np.stack([product(a, b)[0] for a, b in zip(va, vb)])
        assert_equal(y.t, want, f"rows {rows}")


def test_weight_gradients_accumulate_and_leave_empty_groups():
    rows, N, K = [40, 0, 17], 48, 64
    dy = np.concatenate([exact_bits(N, r, i).T for i, r in enumerate(rows) if r])
    x = np.concatenate([exact_bits(K, r, 9 + i).T for i, r in enumerate(rows) if r])
    ga = mx.mx_quantize_grouped(to_dev(dy), rows, axis=mx.COLWISE)
    gb = mx.mx_quantize_grouped(to_dev(x), rows, axis=mx.COLWISE)
    start = torch.randint(-50, 50, (3, N, K), device="cuda").float()
    y = start.clone()
    mx.mx_matmul_wgrad_grouped(ga["q_col"], ga["s_col"], gb["q_col"], gb["s_col"], rows,
                               flags=mx.OUT_F32 | mx.ACCUMULATE, out=y)
    va = split(ga["q_col"], ga["s_col"], [(N, r) for r in rows], 0, False)
    vb = split(gb["q_col"], gb["s_col"], [(K, r) for r in rows], 0, False)
    want = start.cpu().double().numpy() + np.stack([product(a, b)[0] for a, b in zip(va, vb)])
    assert_equal(y, want, "accumulated")
    assert torch.equal(y[1], start[1])


def test_weight_gradient_is_the_derivative():
    """y is linear in W: moving one element of W by d moves sum(y * dY) by
    d * dW[n][k], exactly on exact operands.  Checked against the kernel's own
    forward products of the two weights."""
    M, N, K = 96, 80, 64
    dy, x = exact_bits(N, M, 1).T.copy(), exact_bits(K, M, 2).T.copy()
    w = exact_bits(N, K, 3)
    cd, cx = mx.mx_quantize(to_dev(dy)), mx.mx_quantize(to_dev(x))
    dw = mx.mx_matmul(cd["q_col"], cd["s_col"], cx["q_col"], cx["s_col"], flags=mx.OUT_F32).double()
    gy = torch.from_numpy(mx_values(cd["q_col"], cd["s_col"], N, M)).cuda().t()   # [M][N]
    xr = mx.mx_quantize(to_dev(mx_bits(cx, K, M)), axis=mx.ROWWISE)
    qw, sw = cast_rows(w, 0, False)
    base = mx.mx_matmul(xr["q_row"], xr["s_row"], qw, sw, flags=mx.OUT_F32).double()
    rng = np.random.default_rng(4)
    v0 = mx_values(qw, sw, N, K)
    for _ in range(6):
        n, k = int(rng.integers(N)), int(rng.integers(K))
        q2 = qw.clone()
        q2[n, k] = 0x30                # 0.5: another exact element
        d = mx_values(q2, sw, N, K)[n, k] - v0[n, k]
        moved = mx.mx_matmul(xr["q_row"], xr["s_row"], q2, sw, flags=mx.OUT_F32).double()
        assert ((moved - base) * gy).sum().item() == d * dw[n, k].item()


def mx_bits(cast, K, M):
    """bf16 bits [M][K] of the values a column-wise cast holds."""
    return W.bf16_bits(mx_values(cast["q_col"], cast["s_col"], K, M).T.astype(np.float32))


def test_moe_layer_forward_and_backward():
    """The casts and products of an MoE feed-forward layer together: up
    projection, SwiGLU, down projection, and their gradients, each stage checked
    in 64 bits on the operands the stage before it produced."""
    rows, D, H = [50, 0, 130, 16, 61], 192, 128
    M, G, tile = sum(rows), len(rows), mx.SCALE_TILED
    x, dout = W.normal(M, D, 1), W.normal(M, D, 2)
    w1, w2 = W.normal(G * 2 * H, D, 3, 0.1), W.normal(G * D, H, 4, 0.1)
    c1 = mx.mx_quantize_grouped(to_dev(w1), [2 * H] * G, axis=3 | tile)
    c2 = mx.mx_quantize_grouped(to_dev(w2), [D] * G, axis=3 | tile)
    cx = mx.mx_quantize_grouped(to_dev(x), rows, axis=3 | tile)

    def check(y, qa, sa, sha, qb, sb, shb, ea, what):
        va, vb = split(qa, sa, sha, tile, ea), split(qb, sb, shb, tile, False)
        p = [product(a, b) for a, b in zip(va, vb)]
        cat = np.concatenate if y.dim() == 2 else np.stack
        terms = max(max(s[1] for s in sha), 1)
        assert_close(y, cat([w for w, _ in p]), cat([m for _, m in p]), terms, what,
                     cut=y.dtype == torch.bfloat16)

    def bits(y):
        return y.view(torch.int16)

    h = mx.mx_matmul_grouped(cx["q_row"], cx["s_row"], c1["q_row"], c1["s_row"], rows, flags=tile)
    check(h, cx["q_row"], cx["s_row"], [(r, D) for r in rows], c1["q_row"], c1["s_row"],
          [(2 * H, D)] * G, False, "up")
    ca = mx.mx_quantize_gated_grouped(bits(h), rows, mx.GATED_SWIGLU, axis=3 | tile)
    y = mx.mx_matmul_grouped(ca["q_row"], ca["s_row"], c2["q_row"], c2["s_row"], rows, flags=tile)
    check(y, ca["q_row"], ca["s_row"], [(r, H) for r in rows], c2["q_row"], c2["s_row"],
          [(D, H)] * G, False, "down")
    e5 = mx.ELEM_E5M2
    cd = mx.mx_quantize_grouped(to_dev(dout), rows, axis=3 | tile | e5)
    fl = tile | mx.A_E5M2
    da = mx.mx_matmul_grouped(cd["q_row"], cd["s_row"], c2["q_col"], c2["s_col"], rows, flags=fl)
    check(da, cd["q_row"], cd["s_row"], [(r, D) for r in rows], c2["q_col"], c2["s_col"],
          [(H, D)] * G, True, "down input gradient")
    dw2 = mx.mx_matmul_wgrad_grouped(cd["q_col"], cd["s_col"], ca["q_col"], ca["s_col"], rows,
                                     flags=fl | mx.OUT_F32)
    check(dw2, cd["q_col"], cd["s_col"], [(D, r) for r in rows], ca["q_col"], ca["s_col"],
          [(H, r) for r in rows], True, "down weight gradient")
    ch = mx.mx_quantize_gated_grouped(bits(h), rows, mx.GATED_SWIGLU, grad=bits(da),
                                      axis=3 | tile | e5)
    dx = mx.mx_matmul_grouped(ch["q_row"], ch["s_row"], c1["q_col"], c1["s_col"], rows, flags=fl)
    check(dx, ch["q_row"], ch["s_row"], [(r, 2 * H) for r in rows], c1["q_col"], c1["s_col"],
          [(D, 2 * H)] * G, True, "up input gradient")
    dw1 = mx.mx_matmul_wgrad_grouped(ch["q_col"], ch["s_col"], cx["q_col"], cx["s_col"], rows,
                                     flags=fl | mx.OUT_F32)
    check(dw1, ch["q_col"], ch["s_col"], [(2 * H, r) for r in rows], cx["q_col"], cx["s_col"],
          [(D, r) for r in rows], True, "up weight gradient")
    assert not bool(dw1[1].any()) and not bool(dw2[1].any())


def test_another_stream_and_repeats():
    M, N, K = 300, 520, 1024
    qa, sa, qb, sb, a, b = dense(M, N, K, 0, False, False, seed=71, bits=W.loguniform_rows)
    first = mx.mx_matmul(qa, sa, qb, sb)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ys = [mx.mx_matmul(qa, sa, qb, sb, stream=s) for _ in range(4)]
    s.synchronize()
    assert all(torch.equal(first, y) for y in ys)


def test_captured_products():
    """Graph replays, with new inputs and eager work between them, give the
    eager calls' results."""
    rows, N, K = [100, 0, 33, 64], 256, 320
    M, G = sum(rows), len(rows)
    xs = [to_dev(W.normal(M, K, s)) for s in (1, 2, 3)]
    gs = [to_dev(W.normal(M, N, s)) for s in (4, 5, 6)]
    w = mx.mx_quantize_grouped(to_dev(W.normal(G * N, K, 7)), [N] * G, axis=mx.ROWWISE)
    x, g = xs[0].clone(), gs[0].clone()

    def step():
        cx = mx.mx_quantize_grouped(x, rows)
        cg = mx.mx_quantize_grouped(g, rows)
        y = mx.mx_matmul_grouped(cx["q_row"], cx["s_row"], w["q_row"], w["s_row"], rows)
        dw = mx.mx_matmul_wgrad_grouped(cg["q_col"], cg["s_col"], cx["q_col"], cx["s_col"], rows,
                                        flags=mx.OUT_F32)
        return y, dw

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dw = step()
    for i in (1, 2, 0, 2):
        x.copy_(xs[i])
        g.copy_(gs[i])
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), dw.clone()
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
