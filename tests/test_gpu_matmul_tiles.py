"""MXFP8 products at sizes that take the tiled kernels: whole rounds of 256 x 256
tiles, the last tiles in parts of 128 x 128 or 256 x 128, tiles of 128 x 128, rows
copied to 128-byte boundaries, operands and outputs past 2^32 bytes.

Operands are exact ones (see product_util), made on the GPU as codes and scale
bytes: elements n in {-4 .. 4} and scales 2^-1 .. 2^1, so an output must equal the
float64 product rounded once.  Rows that a tile layout's last tile has too many
hold the NaN byte; blocks it has too many hold 0, as the casts write them.
"""
import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from product_util import E4M3, E5M2, Guarded

pytestmark = pytest.mark.gpu

DT = {0: torch.bfloat16, mx.OUT_F32: torch.float32}
VALUES = np.arange(-4.0, 5.0)


def codes_of(table):
    return np.array([int(np.where(table == v)[0][0]) for v in VALUES], dtype=np.uint8)


def tiled_layout(s):
    """Scale bytes [rows][nb] in the tile layout."""
    rows, nb = s.shape
    RT, CT = -(-rows // 32), -(-nb // 8)
    p = torch.full((RT * 32, CT * 8), 255, dtype=torch.uint8, device=s.device)
    p[:, nb:] = 0
    p[:rows, :nb] = s
    return p.view(RT, 32, CT, 4, 2).permute(2, 0, 4, 1, 3).contiguous().view(-1)


class Operand:
    """Groups of exact rows, one group after the other: codes, scale bytes and
    the float64 values of any rows."""

    def __init__(self, shapes, flags, e5m2, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        table = codes_of(E5M2 if e5m2 else E4M3)
        self.table = torch.from_numpy(table).cuda()
        qs, ss, self.groups = [], [], []
        for rows, K in shapes:
            n = torch.randint(0, 9, (rows, K), device="cuda", dtype=torch.uint8, generator=gen)
            e = torch.randint(126, 129, (rows, -(-K // 32)), device="cuda", dtype=torch.uint8,
                              generator=gen)
            self.groups.append((n, e))
            q = torch.empty_like(n)
            for i in range(0, rows, 65536):          # bounds the index tensor
                q[i:i + 65536] = self.table[n[i:i + 65536].int()]
            qs.append(q.view(-1))
            ss.append(tiled_layout(e) if flags & mx.SCALE_TILED and e.numel() else e.view(-1))
        self.q = torch.cat(qs) if len(qs) > 1 else qs[0]
        self.s = torch.cat(ss) if len(ss) > 1 else ss[0]

    def values(self, g=0, rows=slice(None)):
        n, e = (t[rows] for t in self.groups[g])
        v = (n.double() - 4) * torch.exp2(e.double() - 127).repeat_interleave(32, 1)[:, :n.shape[1]]
        return v


def assert_same(got, want64, what):
    want = want64.float().to(got.dtype)
    same = got == want
    if not bool(same.all()):
        bad = (~same).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {len(bad)} of {same.numel()} differ, first at {i}: "
                             f"{got[i].item()} for {want[i].item()}; last at {bad[-1].tolist()}")


def fmt_flags(ea, eb):
    return (mx.A_E5M2 if ea else 0) | (mx.B_E5M2 if eb else 0)


# (M, N, K): tiles of 128 x 128 (few tiles, short sums), odd and unaligned rows; then
# parts only, whole rounds and parts, halves, one partial round of whole tiles.
SIZES = [(1500, 1301, 2064), (4200, 4157, 400), (6200, 8300, 144), (3800, 3800, 208),
         (4096, 4096, 512), (257, 16500, 1040), (16501, 259, 528), (5000, 4999, 64), (4999, 5000, 32),
         (2500, 2300, 2065), (2049, 4095, 1151), (4200, 4157, 330), (700, 9000, 4001),
         (1500, 1301, 4112), (4200, 4157, 656), (6200, 8300, 640), (5000, 4700, 656),
         (3800, 3801, 784), (4200, 4158, 801), (5000, 4700, 657)]
FORMAT_SIZES = [(1500, 1301, 2064), (2500, 2302, 2065), (4200, 4157, 656), (5000, 4700, 657)]
GROUPED = [([1000, 0, 1, 700, 257, 256], 2500, 1040), ([0, 3000, 0], 4050, 1041),
           ([100] * 40, 4096, 512), ([33, 2900, 5, 0], 3999, 2063),
           ([3000, 0, 1, 700, 257, 256], 4096, 1040)]
WGRAD = [([1000, 0, 1, 700, 257, 256], 2000, 2500), ([512, 2048, 0, 16], 2100, 2300),
         ([1, 2, 3, 2000], 2999, 2111), ([128] * 30, 1200, 2048), ([31, 0, 1808, 640], 3777, 2050)]

@pytest.mark.parametrize("out", [0, mx.OUT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_tiles(M, N, K, tiled, out):
    flags = tiled | out
    a, b = Operand([(M, K)], flags, False, 1), Operand([(N, K)], flags, False, 2)
    y = Guarded((M, N), DT[out])
    mx.mx_matmul(a.q.view(M, K), a.s, b.q.view(N, K), b.s, flags=flags, out=y.t)
    torch.cuda.synchronize()
    y.check("mx_matmul")
    assert_same(y.t, a.values() @ b.values().t(), f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", FORMAT_SIZES)
@pytest.mark.parametrize("ea,eb", [(True, False), (False, True), (True, True)])
def test_tiles_of_every_format(M, N, K, ea, eb):
    for flags in (0, mx.SCALE_TILED, mx.OUT_F32, mx.OUT_F32 | mx.SCALE_TILED):
        f = flags | fmt_flags(ea, eb)
        a, b = Operand([(M, K)], f, ea, 3), Operand([(N, K)], f, eb, 4)
        y = mx.mx_matmul(a.q.view(M, K), a.s, b.q.view(N, K), b.s, flags=f)
        assert_same(y, a.values() @ b.values().t(), f"{M}x{N}x{K} {f}")


@pytest.mark.parametrize("M,N,K", [(1500, 1301, 2064), (1500, 1302, 2064), (4200, 4157, 656),
                                   (4200, 4158, 656)])
def test_tiles_accumulate(M, N, K):
    a, b = Operand([(M, K)], 0, False, 5), Operand([(N, K)], 0, False, 6)
    start = torch.randint(-100, 100, (M, N), device="cuda").float()
    y = Guarded((M, N), torch.float32)
    y.t.copy_(start)
    for _ in range(2):
        mx.mx_matmul(a.q.view(M, K), a.s, b.q.view(N, K), b.s, flags=mx.OUT_F32 | mx.ACCUMULATE,
                     out=y.t)
    torch.cuda.synchronize()
    y.check("accumulate")
    assert_same(y.t, start.double() + 2 * (a.values() @ b.values().t()), "accumulate")


@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("rows,N,K", GROUPED)
def test_grouped_tiles(rows, N, K, tiled):
    G, M = len(rows), sum(rows)
    for flags in (tiled, tiled | mx.OUT_F32 | mx.A_E5M2):
        a = Operand([(r, K) for r in rows], flags, bool(flags & mx.A_E5M2), 7)
        b = Operand([(N, K)] * G, flags, False, 8)
        y = Guarded((M, N), DT[flags & mx.OUT_F32])
        mx.mx_matmul_grouped(a.q.view(M, K), a.s, b.q.view(G * N, K), b.s, rows, flags=flags,
                             out=y.t)
        torch.cuda.synchronize()
        y.check("grouped")
        want = torch.cat([a.values(g) @ b.values(g).t() for g in range(G)])
        assert_same(y.t, want, f"rows {rows}")


@pytest.mark.parametrize("tiled", [0, mx.SCALE_TILED], ids=["compact", "tiled"])
@pytest.mark.parametrize("rows,N,K", WGRAD)
def test_weight_gradient_tiles(rows, N, K, tiled):
    G, M = len(rows), sum(rows)
    for flags in (tiled, tiled | mx.OUT_F32 | mx.A_E5M2):
        a = Operand([(N, r) for r in rows], flags, bool(flags & mx.A_E5M2), 9)
        b = Operand([(K, r) for r in rows], flags, False, 10)
        y = Guarded((G, N, K), DT[flags & mx.OUT_F32])
        mx.mx_matmul_wgrad_grouped(a.q, a.s, b.q, b.s, rows, flags=flags, out=y.t)
        torch.cuda.synchronize()
        y.check("weight gradient")
        want = torch.stack([a.values(g) @ b.values(g).t() for g in range(G)])
        assert_same(y.t, want, f"rows {rows}")


@pytest.mark.parametrize("M,N,K,flags", [
    (262165, 40, 16400, 0),                          # A past 2^32 bytes
    (40, 262165, 16400, mx.SCALE_TILED),             # B
    (66000, 33000, 48, mx.OUT_F32),                  # the output
    (20, 8200, 524304, 0),                           # B, small products' kernel
    (262165, 270, 16401, mx.SCALE_TILED)])            # A's copy
def test_past_32_bits(M, N, K, flags):
    """Sums of up to 524304 exact products stay below 2^24 quarters here: they
    have random signs and a standard deviation of less than 12000."""
    a, b = Operand([(M, K)], flags, False, 11), Operand([(N, K)], flags, False, 12)
    y = mx.mx_matmul(a.q.view(M, K), a.s, b.q.view(N, K), b.s, flags=flags)
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(13)
    mi = torch.cat([torch.tensor([0, M - 1]), torch.randint(0, M, (30,), generator=gen)]).cuda()
    ni = torch.cat([torch.tensor([0, N - 1]), torch.randint(0, N, (30,), generator=gen)]).cuda()
    va, vb = a.values(rows=mi), b.values(rows=ni)
    assert_same(y[mi][:, ni], va @ vb.t(), "sampled")
    if K < 20000:
        for i in range(0, 32, 8):                    # whole rows and columns
            r = mi[i:i + 8]
            if N < 100:
                assert_same(y[r], a.values(rows=r) @ b.values().t(), "rows")
            if M < 100:
                assert_same(y[:, ni[i:i + 8]], a.values() @ b.values(rows=ni[i:i + 8]).t(), "columns")


def test_own_workspaces_on_two_streams():
    """Two packed products at a time, each with its own workspace, and the given
    workspace's bytes behind the needed ones untouched."""
    M, N, K = 2500, 2300, 2065
    need = mx.mx_matmul_workspace_size(M, N, K)
    assert need == (M + N) * 2176
    ops = [(Operand([(M, K)], 0, False, 20 + i), Operand([(N, K)], 0, False, 30 + i)) for i in range(2)]
    want = [(a.values() @ b.values().t()).float().bfloat16() for a, b in ops]
    ws = [torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda") for _ in ops]
    streams = [torch.cuda.Stream() for _ in ops]
    ys = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in ops]
    torch.cuda.synchronize()
    for _ in range(3):
        for (a, b), w, s, y in zip(ops, ws, streams, ys):
            mx.mx_matmul(a.q.view(M, K), a.s, b.q.view(N, K), b.s, out=y, workspace=w, stream=s)
    torch.cuda.synchronize()
    for y, w, v in zip(ys, ws, want):
        assert torch.equal(y, v)
        assert bool((w[need:] == 0xA5).all())


def test_captured_with_a_copy_of_the_rows():
    """Graph replays of a packed product and weight gradient, with new operands
    and eager work between them."""
    rows, N, K = [1000, 0, 333, 767], 2100, 2500
    M, G = sum(rows), len(rows)
    sets = [(Operand([(N, r) for r in rows], 0, False, 40 + i),
             Operand([(K, r) for r in rows], 0, False, 50 + i)) for i in range(3)]
    a, sa, b, sb = (t.clone() for t in (sets[0][0].q, sets[0][0].s, sets[0][1].q, sets[0][1].s))
    assert mx.mx_matmul_wgrad_grouped_workspace_size(N, K, rows) > 0

    def step():
        return mx.mx_matmul_wgrad_grouped(a, sa, b, sb, rows, flags=mx.OUT_F32)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for i in (1, 2, 0, 2):
        for t, v in zip((a, sa, b, sb), (sets[i][0].q, sets[i][0].s, sets[i][1].q, sets[i][1].s)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.stack([sets[i][0].values(g) @ sets[i][1].values(g).t() for g in range(G)])
        assert_same(y, want, f"replay of {i}")
        assert torch.equal(step(), y)
