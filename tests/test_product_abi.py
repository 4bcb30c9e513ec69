"""Contract of the products' entry points that needs no GPU: every malformed
call is refused with its status before any memory is touched, the workspace
sizes, and the binding's own checks (which run before the device check, so CPU
tensors reach them)."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_precision_bf16_amd as mx

U8, F32, BF16, I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


class Host:
    """16-byte aligned host buffers standing in for device memory, with canaries."""

    def __init__(self, **sizes):
        self.raw = {k: np.full(n + 64, 0xA5, np.uint8) for k, n in sizes.items()}

    def p(self, name, shift=0):
        a = self.raw[name]
        return a.ctypes.data + (-a.ctypes.data) % 16 + shift

    def untouched(self):
        return all(np.all(a == 0xA5) for a in self.raw.values())


M, N, K = 64, 96, 128


def mm(h, qa=None, sa=None, qb=None, sb=None, m=M, n=N, k=K, flags=0, y=None, ws=None, wn=0):
    g = lambda v, name: h.p(name) if v is None else v
    return mx.lib().mx_matmul(g(qa, "qa"), g(sa, "sa"), g(qb, "qb"), g(sb, "sb"), m, n, k, flags,
                              g(y, "y"), ws, wn, None)


@pytest.fixture
def h():
    return Host(qa=M * K, sa=M * K // 32, qb=N * K, sb=N * K // 32, y=4 * M * N, ws=4096)


def test_product_errors(h):
    assert mm(h, flags=1) == mx.MX_ERR_ENUM
    assert mm(h, flags=8) == mx.MX_ERR_ENUM
    assert mm(h, flags=256) == mx.MX_ERR_ENUM
    assert mm(h, flags=mx.ACCUMULATE) == mx.MX_ERR_ENUM          # needs OUT_F32
    for name in ("qa", "sa", "qb", "sb", "y"):
        assert mm(h, **{name: 0}) == mx.MX_ERR_NULL
        assert mm(h, **{name: h.p(name, 8)}) == mx.MX_ERR_ALIGN
    for bad in (0, -1, (1 << 23) + 1, 1 << 62, -(1 << 62)):
        assert mm(h, m=bad) == mx.MX_ERR_SHAPE
        assert mm(h, n=bad) == mx.MX_ERR_SHAPE
        assert mm(h, k=bad) == mx.MX_ERR_SHAPE
    assert mm(h, m=1 << 22, n=1 << 22) == mx.MX_ERR_SHAPE        # 2^44 outputs
    for name in ("qa", "sa", "qb", "sb"):
        assert mm(h, y=h.p(name)) == mx.MX_ERR_ALIAS
    assert h.untouched()


def test_workspace(h):
    """Operands whose rows do not start at multiples of 16 bytes need copies with
    rows of whole 128-byte lines, unless the product is small."""
    size = mx.mx_matmul_workspace_size
    assert size(8192, 8192, 8192) == 0 and size(64, 64, 33) == 0
    assert size(4096, 4096, 4095) == 2 * 4096 * 4096
    assert size(4096, 4096, 4104) == 2 * 4096 * 4224
    assert size(0, 64, 64) == 0 and size(64, 64, 64, 1) == 0
    assert mx.mx_matmul_grouped_workspace_size(2048, 4000, [4096, 0, 100]) == 0
    assert mx.mx_matmul_grouped_workspace_size(2048, 4001, [4096, 0, 100]) == \
        (4196 + 3 * 2048) * 4096
    assert mx.mx_matmul_wgrad_grouped_workspace_size(2048, 5120, [2000, 0, 4000]) == 0
    assert mx.mx_matmul_wgrad_grouped_workspace_size(2048, 5120, [2001, 0, 4000]) == \
        (2048 + 5120) * (2048 + 4096)
    big = Host(qa=16, sa=16, qb=16, sb=16, y=16)
    args = dict(m=4096, n=4096, k=4095)
    assert mm(big, **args) == mx.MX_ERR_WORKSPACE
    far = 1 << 40                    # addresses far from each other, never read
    spread = dict(qa=far, sa=2 * far, qb=3 * far, sb=4 * far, y=5 * far)
    assert mm(big, **args, **spread, ws=6 * far, wn=2 * 4096 * 4096 - 1) == mx.MX_ERR_WORKSPACE
    assert mm(big, **args, **spread, ws=6 * far + 8, wn=1 << 30) == mx.MX_ERR_ALIGN
    for at in spread.values():
        assert mm(big, **args, **spread, ws=at, wn=1 << 30) == mx.MX_ERR_ALIAS
    assert big.untouched()


def grouped(h, rows, fn="mx_matmul_grouped", n=N, k=K, G=None):
    arr = (ctypes.c_int64 * max(len(rows), 1))(*rows)
    return getattr(mx.lib(), fn)(h.p("qa"), h.p("sa"), h.p("qb"), h.p("sb"), n, k,
                                 ctypes.addressof(arr), len(rows) if G is None else G, 0, h.p("y"),
                                 None, 0, None)


@pytest.mark.parametrize("fn", ["mx_matmul_grouped", "mx_matmul_wgrad_grouped"])
def test_group_errors(h, fn):
    assert grouped(h, [], fn) == mx.MX_ERR_SHAPE
    assert grouped(h, [1] * 65, fn) == mx.MX_ERR_SHAPE
    assert grouped(h, [0, 0], fn) == mx.MX_ERR_SHAPE
    assert grouped(h, [16, -16, 16], fn) == mx.MX_ERR_SHAPE
    assert grouped(h, [1 << 23, 1], fn) == mx.MX_ERR_SHAPE
    assert grouped(h, [1 << 62, 1 << 62], fn) == mx.MX_ERR_SHAPE
    assert grouped(h, [64], fn, G=-1) == mx.MX_ERR_SHAPE
    assert grouped(h, [64], fn, n=0) == mx.MX_ERR_SHAPE
    assert grouped(h, [64], fn, k=-5) == mx.MX_ERR_SHAPE
    L = mx.lib()
    assert getattr(L, fn)(h.p("qa"), h.p("sa"), h.p("qb"), h.p("sb"), N, K, None, 1, 0, h.p("y"), None,
                          0, None) == mx.MX_ERR_NULL
    assert h.untouched()


def test_matvec_errors():
    T, top, G = 4, 2, 3
    h = Host(x=2 * T * K, e=4 * T * top, qw=G * N * K // 2, sw=G * N * K // 16, sg=64,
             y=4 * T * top * N)
    L = mx.lib()

    def mv(x=None, qw=None, sw=None, sg=None, y=None, t=T, n=N, k=K, flags=0):
        g = lambda v, name: h.p(name) if v is None else v
        return L.nvfp4_matvec(g(x, "x"), t, g(qw, "qw"), g(sw, "sw"), g(sg, "sg"), n, k, flags,
                              g(y, "y"), None)

    def ex(e=None, t=T, tp=top, g_=G, n=N, k=K, y=None, flags=0):
        return L.nvfp4_matvec_experts(h.p("x"), h.p("e") if e is None else e, t, tp, h.p("qw"),
                                      h.p("sw"), h.p("sg"), g_, n, k, flags, h.p("y") if y is None
                                      else y, None)

    for flags in (1, mx.ACCUMULATE | mx.OUT_F32, mx.SCALE_TILED):
        assert mv(flags=flags) == mx.MX_ERR_ENUM and ex(flags=flags) == mx.MX_ERR_ENUM
    for name in ("x", "qw", "sw", "sg", "y"):
        assert mv(**{name: 0}) == mx.MX_ERR_NULL
    for name in ("x", "qw", "sw", "y"):
        assert mv(**{name: h.p(name, 4)}) == mx.MX_ERR_ALIGN
    assert mv(sg=h.p("sg", 2)) == mx.MX_ERR_ALIGN
    for name in ("x", "qw", "sw", "sg"):
        assert mv(y=h.p(name)) == mx.MX_ERR_ALIAS
    for bad in (0, -3, (1 << 23) + 1, 1 << 62):
        assert mv(t=bad) == mx.MX_ERR_SHAPE and mv(n=bad) == mx.MX_ERR_SHAPE
        assert mv(k=bad) == mx.MX_ERR_SHAPE and ex(t=bad) == mx.MX_ERR_SHAPE
    assert ex(e=0) == mx.MX_ERR_NULL and ex(e=h.p("e", 2)) == mx.MX_ERR_ALIGN
    assert ex(tp=0) == mx.MX_ERR_SHAPE and ex(tp=65) == mx.MX_ERR_SHAPE
    assert ex(t=1 << 23, tp=2) == mx.MX_ERR_SHAPE
    assert ex(g_=0) == mx.MX_ERR_SHAPE and ex(g_=1025) == mx.MX_ERR_SHAPE
    assert ex(g_=1024, n=1 << 20, k=1 << 20) == mx.MX_ERR_SHAPE
    assert ex(y=h.p("e")) == mx.MX_ERR_ALIAS
    assert h.untouched()


def z(*shape, dtype=U8):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call,exc,match", [
    (lambda: mx.mx_matmul(z(4, 64, dtype=F32), z(8), z(4, 64), z(8)), TypeError, "qa"),
    (lambda: mx.mx_matmul(z(4, 128)[:, :64], z(8), z(4, 64), z(8)), ValueError, "contiguous"),
    (lambda: mx.mx_matmul(z(4, 64), z(8), z(4, 32), z(4)), ValueError, "one K"),
    (lambda: mx.mx_matmul(z(4, 64), z(9), z(4, 64), z(8)), ValueError, "sa must have 8"),
    (lambda: mx.mx_matmul(z(4, 64), z(8), z(4, 64), z(8), flags=mx.SCALE_TILED), ValueError,
     "sa must have 256"),
    (lambda: mx.mx_matmul(z(4, 64), z(8), z(4, 64), z(8), out=z(4, 4, dtype=F32)), ValueError, "out must"),
    (lambda: mx.mx_matmul(z(4, 64), z(8), z(4, 64), z(8), flags=mx.OUT_F32, out=z(4, 4, dtype=BF16)),
     ValueError, "out must"),
    (lambda: mx.mx_matmul(z(4, 64), z(8), z(4, 64), z(8), out=z(4, 5, dtype=BF16)), ValueError, "out must"),
    (lambda: mx.mx_matmul(z(4, 64), z(8), z(4, 64), z(8), flags=mx.OUT_F32 | mx.ACCUMULATE), ValueError,
     "ACCUMULATE"),
    (lambda: mx.mx_matmul_grouped(z(6, 64), z(12), z(2, 4, 64), z(16), [4, 1]), ValueError, "sum"),
    (lambda: mx.mx_matmul_grouped(z(6, 64), z(12), z(2, 4, 63), z(16), [4, 2]), ValueError, "2 matrices"),
    (lambda: mx.mx_matmul_grouped(z(6, 64), z(12), z(2, 4, 64), z(15), [4, 2]), ValueError, "sb must"),
    (lambda: mx.mx_matmul_wgrad_grouped(z(6 * 8), z(16), z(6 * 4 + 1), z(8), [4, 2]), ValueError, "columns"),
    (lambda: mx.mx_matmul_wgrad_grouped(z(6 * 8), z(15), z(6 * 4), z(8), [4, 2]), ValueError, "sa must"),
    (lambda: mx.mx_matmul_wgrad_grouped(z(0), z(0), z(0), z(0), [0, 0]), ValueError, "columns"),
    (lambda: mx.nvfp4_matvec(z(2, 64, dtype=F32), z(4, 32), z(4, 4), z(1, dtype=F32)), TypeError, "bf16"),
    (lambda: mx.nvfp4_matvec(z(2, 64, dtype=BF16), z(4, 31), z(4, 4), z(1, dtype=F32)), ValueError, "qw must"),
    (lambda: mx.nvfp4_matvec(z(2, 64, dtype=BF16), z(4, 32), z(4, 3), z(1, dtype=F32)), ValueError, "sw must"),
    (lambda: mx.nvfp4_matvec(z(2, 64, dtype=BF16), z(4, 32), z(4, 4), z(2, dtype=F32)), ValueError, "sg must"),
    (lambda: mx.nvfp4_matvec_experts(z(2, 64, dtype=BF16), z(2, 2, dtype=torch.int64), z(8, 32), z(8, 4),
                                     z(2, dtype=F32)), ValueError, "experts"),
    (lambda: mx.nvfp4_matvec_experts(z(2, 64, dtype=BF16), z(3, 2, dtype=I32), z(8, 32), z(8, 4),
                                     z(2, dtype=F32)), ValueError, "experts"),
    (lambda: mx.nvfp4_matvec_experts(z(2, 64, dtype=BF16), z(2, 2, dtype=I32), z(9, 32), z(9, 4),
                                     z(2, dtype=F32)), ValueError, "2 matrices"),
])
def test_binding_refusals(call, exc, match):
    with pytest.raises(exc, match=match):
        call()


@pytest.mark.parametrize("call", [
    lambda: mx.mx_matmul(z(4, 64), z(8), z(4, 64), z(8)),
    lambda: mx.mx_matmul_grouped(z(6, 64), z(12), z(2, 4, 64), z(16), [4, 2]),
    lambda: mx.mx_matmul_wgrad_grouped(z(6 * 8), z(16), z(6 * 4), z(8), [4, 2]),
    lambda: mx.nvfp4_matvec(z(2, 64, dtype=BF16), z(4, 32), z(4, 4), z(1, dtype=F32)),
    lambda: mx.nvfp4_matvec_experts(z(2, 64, dtype=BF16), z(2, 2, dtype=I32), z(8, 32), z(8, 4),
                                    z(2, dtype=F32)),
], ids=["matmul", "grouped", "wgrad", "matvec", "experts"])
def test_host_tensors_never_reach_the_library(call):
    with pytest.raises(ValueError, match="ROCm"):
        call()
