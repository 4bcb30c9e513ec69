"""Contract of the norm's, the router's and the rows' entry points that needs no
GPU: every malformed call is refused with its status before any memory is touched,
workspace sizes, and the binding's own checks (which run before the device check,
so CPU tensors reach them)."""
import ctypes
import math

import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from test_product_abi import Host

BF16, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
BIG = 1 << 40


def call(fn, h, names, values):
    """fn by its C arguments: a name stands for that host buffer unless `values`
    gives it another value."""
    args = []
    for n in names:
        v = values.get(n, n)
        args.append(h.p(v) if isinstance(v, str) and v in h.raw else v)
    return getattr(mx.lib(), fn)(*args, None)


M, K = 48, 96
NORM = ("x", "residual", "weight", "M", "K", "eps", "axis", "h", "y", "q_row", "s_row", "q_col",
        "s_col", "q_h", "s_h", "rstd", "ws", "wn")


@pytest.fixture
def nh():
    n = M * K
    return Host(x=2 * n, residual=2 * n, weight=2 * K, h=2 * n, y=2 * n, q_row=n, s_row=2 * 256,
                q_col=n, s_col=3 * 256, q_h=n, s_h=M * 3, rstd=4 * M, ws=8 * M)


def norm(host, /, **kw):
    return call("mx_rmsnorm", host, NORM, dict(M=M, K=K, eps=1e-6, axis=3, wn=8 * M) | kw)


def test_norm_errors(nh):
    for axis in (4, 8, 16, 32, 1 | 32, 1 << 31):
        assert norm(nh, axis=axis) == mx.MX_ERR_ENUM
    for eps in (-1e-6, math.inf, math.nan, -math.inf):
        assert norm(nh, eps=eps) == mx.MX_ERR_ENUM
    for name in ("x", "h", "q_row", "s_row", "q_col", "s_col", "q_h", "s_h", "rstd"):
        assert norm(nh, **{name: None}) == mx.MX_ERR_NULL, name
    for bad in (0, -1, (1 << 23) + 1, 1 << 62, -(1 << 62)):
        assert norm(nh, M=bad) == mx.MX_ERR_SHAPE
        assert norm(nh, K=bad) == mx.MX_ERR_SHAPE
    assert norm(nh, M=1 << 22, K=1 << 22) == mx.MX_ERR_SHAPE
    for name in NORM:
        if name in nh.raw:
            assert norm(nh, **{name: nh.p(name, 8)}) == mx.MX_ERR_ALIGN, name
    assert norm(nh, ws=None) == mx.MX_ERR_WORKSPACE and norm(nh, wn=8 * M - 1) == mx.MX_ERR_WORKSPACE
    assert norm(nh, axis=2, ws=None, wn=0) == mx.MX_ERR_WORKSPACE
    size = mx.mx_rmsnorm_workspace_size
    assert size(M, 3) == size(M, 2) == 8 * M and size(M, 1) == size(M, 0) == size(0, 2) == size(-1, 2) == 0
    outputs = ("h", "y", "q_row", "s_row", "q_col", "s_col", "q_h", "s_h", "rstd", "ws")
    for o in outputs:
        for i in ("x", "residual", "weight") + tuple(p for p in outputs if p != o):
            assert norm(nh, **{o: nh.p(i)}) == mx.MX_ERR_ALIAS, (o, i)
    # the tile layout's scales are longer than the compact ones: s_row 512 bytes
    assert norm(nh, axis=1 | mx.SCALE_TILED, rstd=nh.p("s_row", 256)) == mx.MX_ERR_ALIAS
    assert nh.untouched()


BACK = ("dy", "h", "q_h", "s_h", "rstd", "weight", "dres", "M", "K", "dh", "dweight", "ws", "wn")


def back(host, /, **kw):
    return call("mx_rmsnorm_backward", host, BACK, dict(M=M, K=K, q_h=None, s_h=None, wn=1 << 20) | kw)


def test_norm_backward_errors():
    n = M * K
    h = Host(dy=2 * n, h=2 * n, q_h=n, s_h=3 * M, rstd=4 * M, weight=2 * K, dres=2 * n, dh=2 * n,
             dweight=4 * K, ws=4 * K * M)
    for name in ("dy", "h", "rstd", "dh"):
        assert back(h, **{name: None}) == mx.MX_ERR_NULL, name
    assert back(h, q_h="q_h", s_h="s_h") == mx.MX_ERR_NULL            # both
    assert back(h, h=None, q_h="q_h") == mx.MX_ERR_NULL               # codes without scales
    assert back(h, s_h="s_h") == mx.MX_ERR_NULL                       # scales without codes
    for bad in (0, -1, (1 << 23) + 1, 1 << 62):
        assert back(h, M=bad) == mx.MX_ERR_SHAPE
        assert back(h, K=bad) == mx.MX_ERR_SHAPE
    for name in BACK:
        if name in h.raw:
            kw = dict(h=None, q_h="q_h", s_h="s_h") if name in ("q_h", "s_h") else {}
            assert back(h, **kw | {name: h.p(name, 8)}) == mx.MX_ERR_ALIGN, name
    need = mx.mx_rmsnorm_backward_workspace_size(M, K)
    assert need > 0 and need % (4 * K) == 0
    assert back(h, ws=None, wn=0) == mx.MX_ERR_WORKSPACE
    assert back(h, wn=need - 1) == mx.MX_ERR_WORKSPACE
    for o in ("dh", "dweight", "ws"):
        for i in ("dy", "h", "rstd", "weight", "dres"):
            assert back(h, **{o: h.p(i)}) == mx.MX_ERR_ALIAS, (o, i)
        for i in ("q_h", "s_h"):
            assert back(h, h=None, q_h="q_h", s_h="s_h", **{o: h.p(i)}) == mx.MX_ERR_ALIAS, (o, i)
    assert back(h, dh=h.p("dweight")) == mx.MX_ERR_ALIAS
    assert back(h, ws=h.p("dh")) == mx.MX_ERR_ALIAS
    assert h.untouched()


def test_norm_backward_workspace():
    size = mx.mx_rmsnorm_backward_workspace_size
    for m, k in ((0, 8), (8, 0), (-1, 8), ((1 << 23) + 1, 8), (1 << 22, 1 << 22)):
        assert size(m, k) == 0
    assert size(1, 8) == 4 * 8 and size(1, 7) == 4 * 7
    for k in (8, 4096, 8192, 16384, 16385, 1111):
        assert all(size(m, k) <= size(m + 1, k) for m in (1, 7, 255, 300, 1000))
        assert size(1 << 17, k) == size(1 << 18, k)      # a bound number of workgroups


T, E, TOP = 6, 16, 3
ROUTE = ("logits", "bias", "T", "E", "top", "groups", "top_groups", "scale", "flags", "experts",
         "weights", "scores")


def route(h, **kw):
    return call("moe_route", h, ROUTE, dict(T=T, E=E, top=TOP, groups=4, top_groups=2, scale=1.0,
                                            flags=8) | kw)


def test_route_errors():
    h = Host(logits=4 * T * E, bias=4 * E, experts=4 * T * TOP, weights=4 * T * TOP, scores=4 * T * E)
    for flags in (16, 32, 1 << 31):
        assert route(h, flags=flags) == mx.MX_ERR_ENUM
    for scale in (math.inf, -math.inf, math.nan):
        assert route(h, scale=scale) == mx.MX_ERR_ENUM
    for name in ("logits", "experts", "weights"):
        assert route(h, **{name: None}) == mx.MX_ERR_NULL
    for kw in (dict(T=0), dict(T=-1), dict(T=(1 << 23) + 1), dict(E=0), dict(E=-4), dict(E=1028),
               dict(top=0), dict(top=-1), dict(top=17), dict(E=128, top=65), dict(groups=0),
               dict(groups=-1), dict(groups=3), dict(groups=32), dict(E=256, groups=128),
               dict(top_groups=0), dict(top_groups=5), dict(T=1 << 62)):
        assert route(h, **kw) == mx.MX_ERR_SHAPE, kw
    for name in ("logits", "experts", "weights", "scores"):
        assert route(h, **{name: h.p(name, 8)}) == mx.MX_ERR_ALIGN
    assert route(h, bias=h.p("bias", 2)) == mx.MX_ERR_ALIGN
    for o in ("experts", "weights", "scores"):
        for i in ("logits", "bias") + tuple(p for p in ("experts", "weights", "scores") if p != o):
            assert route(h, **{o: h.p(i)}) == mx.MX_ERR_ALIAS, (o, i)
    assert h.untouched()


RBACK = ("logits", "experts", "dweights", "dscores", "T", "E", "top", "scale", "flags", "dlogits")


def test_route_backward_errors():
    h = Host(logits=4 * T * E, experts=4 * T * TOP, dweights=4 * T * TOP, dscores=4 * T * E,
             dlogits=4 * T * E)

    def rb(**kw):
        return call("moe_route_backward", h, RBACK, dict(T=T, E=E, top=TOP, scale=1.0, flags=8) | kw)

    assert rb(flags=16) == mx.MX_ERR_ENUM and rb(scale=math.nan) == mx.MX_ERR_ENUM
    for name in ("logits", "experts", "dweights", "dlogits"):
        assert rb(**{name: None}) == mx.MX_ERR_NULL
    for kw in (dict(T=0), dict(E=0), dict(E=1025), dict(top=0), dict(top=17), dict(T=1 << 24)):
        assert rb(**kw) == mx.MX_ERR_SHAPE, kw
    for name in ("logits", "experts", "dweights", "dscores", "dlogits"):
        assert rb(**{name: h.p(name, 4)}) == mx.MX_ERR_ALIGN
    for i in ("logits", "experts", "dweights", "dscores"):
        assert rb(dlogits=h.p(i)) == mx.MX_ERR_ALIAS
    assert h.untouched()


SORT = ("experts", "T", "top", "E", "align", "rows", "counts", "pos", "slots", "ws", "wn")


def test_sort_errors():
    rows = mx.moe_sort_rows(T, TOP, E, 16)
    assert rows == T * TOP + 16 * 15
    h = Host(experts=4 * T * TOP, counts=4 * E, pos=4 * T * TOP, slots=4 * rows, ws=64)

    def sort(**kw):
        return call("moe_sort", h, SORT, dict(T=T, top=TOP, E=E, align=16, rows=rows, ws=None, wn=0) | kw)

    for name in ("experts", "counts", "pos", "slots"):
        assert sort(**{name: None}) == mx.MX_ERR_NULL
    for kw in (dict(T=0), dict(T=-1), dict(top=0), dict(top=65), dict(E=0), dict(E=1025),
               dict(align=0), dict(align=-1), dict(align=4097), dict(rows=rows - 1), dict(rows=0),
               dict(rows=(1 << 24) + 1), dict(T=1 << 23, top=2), dict(T=1 << 62)):
        assert sort(**kw) == mx.MX_ERR_SHAPE, kw
    for name in ("experts", "counts", "pos", "slots"):
        assert sort(**{name: h.p(name, 4)}) == mx.MX_ERR_ALIGN
        for other in ("experts", "counts", "pos", "slots"):
            if other != name:
                assert sort(**{name: h.p(other)}) == mx.MX_ERR_ALIAS
    # many slots need a workspace
    far = {n: (i + 1) * BIG for i, n in enumerate(("experts", "counts", "pos", "slots"))}
    many = dict(T=65536, top=8, align=1, rows=1 << 20, **far)
    need = mx.moe_sort_workspace_size(65536, 8, E)
    assert need > 0
    assert sort(**many) == mx.MX_ERR_WORKSPACE
    assert sort(**many, ws=9 * BIG) == mx.MX_ERR_WORKSPACE
    assert sort(**many | dict(ws=9 * BIG, wn=need - 1)) == mx.MX_ERR_WORKSPACE
    assert sort(**many | dict(ws=9 * BIG + 4, wn=need)) == mx.MX_ERR_ALIGN
    for at in far.values():
        assert sort(**many | dict(ws=at, wn=need)) == mx.MX_ERR_ALIAS
    assert h.untouched()


def test_sort_sizes():
    rows, size = mx.moe_sort_rows, mx.moe_sort_workspace_size
    assert rows(1, 1, 1024, 4096) == 4096              # one slot: one expert's padding
    assert rows(4096, 4, 8, 16) == 16384 + 8 * 15 and rows(4096, 4, 8, 1) == 16384
    assert rows(1 << 23, 1, 1, 1) == 1 << 23
    for bad in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 65, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                (1, 1, 1, 4097), (1 << 23, 2, 1, 1), (-1, 1, 1, 1)):
        assert rows(*bad) == 0
    assert size(4096, 8, 64) == 0 and size(4097, 8, 64) > 0 and size(0, 8, 64) == 0
    for t in (4097, 1 << 17, 1 << 20):
        blocks = size(t, 8, 64) // 256
        assert 1 <= blocks <= 256 and size(t, 8, 64) == 256 * blocks


def test_gather_errors():
    h = Host(x=64 * T, slots=4 * 20, out=64 * 20)
    names = ("x", "T", "top", "slots", "rows", "row_bytes", "out")

    def gather(**kw):
        return call("moe_gather", h, names, dict(T=T, top=TOP, rows=20, row_bytes=64) | kw)

    for name in ("x", "slots", "out"):
        assert gather(**{name: None}) == mx.MX_ERR_NULL
        assert gather(**{name: h.p(name, 8)}) == mx.MX_ERR_ALIGN
    for kw in (dict(T=0), dict(top=0), dict(top=65), dict(rows=0), dict(rows=(1 << 24) + 1),
               dict(row_bytes=0), dict(row_bytes=(1 << 24) + 1), dict(T=1 << 23, top=2),
               dict(rows=1 << 24, row_bytes=1 << 18)):
        assert gather(**kw) == mx.MX_ERR_SHAPE, kw
    assert gather(out=h.p("x")) == mx.MX_ERR_ALIAS and gather(out=h.p("slots")) == mx.MX_ERR_ALIAS
    assert h.untouched()


def test_combine_errors():
    R = 20
    h = Host(y=2 * R * K, pos=4 * T * TOP, weights=4 * T * TOP, out=2 * T * K, dout=2 * T * K,
             slots=4 * R, dy=2 * R * K, dweights=4 * T * TOP)
    fwd = ("y", "R", "K", "pos", "weights", "T", "top", "out")
    bwd = ("dout", "y", "R", "K", "pos", "slots", "weights", "T", "top", "dy", "dweights")
    size = dict(R=R, K=K, T=T, top=TOP)
    f = lambda **kw: call("moe_combine", h, fwd, size | kw)
    b = lambda **kw: call("moe_combine_backward", h, bwd, size | kw)
    assert f(y=None) == f(out=None) == mx.MX_ERR_NULL
    for name in ("dout", "y", "dy", "pos", "slots"):
        assert b(**{name: None}) == mx.MX_ERR_NULL, name
    for kw in (dict(T=0), dict(top=0), dict(top=65), dict(R=0), dict(K=0), dict(K=-1),
               dict(R=(1 << 24) + 1), dict(K=(1 << 23) + 1), dict(T=1 << 23, top=2),
               dict(R=1 << 24, K=1 << 17)):
        assert f(**kw) == mx.MX_ERR_SHAPE and b(**kw) == mx.MX_ERR_SHAPE, kw
    assert f(pos=None) == mx.MX_ERR_SHAPE                  # 18 slots, 20 rows
    assert b(pos=None, slots=None) == mx.MX_ERR_SHAPE
    for name in ("y", "pos", "weights", "out"):
        assert f(**{name: h.p(name, 8)}) == mx.MX_ERR_ALIGN
    for name in ("dout", "y", "pos", "slots", "weights", "dy", "dweights"):
        assert b(**{name: h.p(name, 8)}) == mx.MX_ERR_ALIGN
    for i in ("y", "pos", "weights"):
        assert f(out=h.p(i)) == mx.MX_ERR_ALIAS
    for o in ("dy", "dweights"):
        for i in ("dout", "y", "pos", "slots", "weights"):
            assert b(**{o: h.p(i)}) == mx.MX_ERR_ALIAS
    assert b(dy=h.p("dweights")) == mx.MX_ERR_ALIAS
    assert h.untouched()


# ---- the binding ---------------------------------------------------------------

def z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


x, ex, lg = z(4, 64), z(4, 2, dtype=I32), z(4, 8, dtype=F32)

WRONG = [
    lambda: mx.mx_rmsnorm(z(4, 64, dtype=F32)),
    lambda: mx.mx_rmsnorm(z(64)),
    lambda: mx.mx_rmsnorm(x.t()),
    lambda: mx.mx_rmsnorm(x, z(32)),
    lambda: mx.mx_rmsnorm(x, z(64, dtype=F32)),
    lambda: mx.mx_rmsnorm(x, residual=z(4, 32)),
    lambda: mx.mx_rmsnorm(x, out=dict(y=z(4, 32))),
    lambda: mx.mx_rmsnorm(x, axis=1, out=dict(s_row=z(4, 3, dtype=U8))),
    lambda: mx.mx_rmsnorm(x, axis=2, workspace=7),
    lambda: mx.mx_rmsnorm(x, axis=2, workspace=z(64, 4).t()),
    lambda: mx.mx_rmsnorm_backward(x, z(4, dtype=F32)),
    lambda: mx.mx_rmsnorm_backward(x, z(4, dtype=F32), h=x, q_h=z(4, 64, dtype=U8),
                                   s_h=z(4, 2, dtype=U8)),
    lambda: mx.mx_rmsnorm_backward(x, z(4, dtype=F32), q_h=z(4, 64, dtype=U8)),
    lambda: mx.mx_rmsnorm_backward(x, z(4, dtype=F32), q_h=z(4, 64, dtype=U8), s_h=z(4, 1, dtype=U8)),
    lambda: mx.mx_rmsnorm_backward(x, z(3, dtype=F32), h=x),
    lambda: mx.mx_rmsnorm_backward(x, z(4, dtype=BF16), h=x),
    lambda: mx.mx_rmsnorm_backward(x, z(4, dtype=F32), h=x, dres=z(4, 32)),
    lambda: mx.moe_route(z(4, 8, dtype=torch.float16), 2),
    lambda: mx.moe_route(z(8), 2),
    lambda: mx.moe_route(lg.t(), 2),
    lambda: mx.moe_route(lg, 2, bias=z(8)),
    lambda: mx.moe_route(lg, 2, bias=z(7, dtype=F32)),
    lambda: mx.moe_route(lg, 2, out=dict(experts=z(4, 3, dtype=I32))),
    lambda: mx.moe_route_backward(z(4, 2), lg, ex),
    lambda: mx.moe_route_backward(z(4, 3, dtype=F32), lg, ex),
    lambda: mx.moe_route_backward(z(4, 2, dtype=F32), lg, ex.long()),
    lambda: mx.moe_route_backward(z(4, 2, dtype=F32), lg, ex, dscores=z(4, 7, dtype=F32)),
    lambda: mx.moe_sort(ex.long(), 8),
    lambda: mx.moe_sort(z(8, dtype=I32), 8),
    lambda: mx.moe_sort(ex, 8, out=dict(counts=z(7, dtype=I32))),
    lambda: mx.moe_gather(x, ex, 2),
    lambda: mx.moe_gather(x, z(8, dtype=torch.int64), 2),
    lambda: mx.moe_gather(x.t(), z(8, dtype=I32), 2),
    lambda: mx.moe_gather(x, z(8, dtype=I32), 2, out=z(8, 32)),
    lambda: mx.moe_combine(x),
    lambda: mx.moe_combine(z(8, 64), weights=z(4, 3, dtype=F32), pos=ex),
    lambda: mx.moe_combine(z(8, 64), weights=z(4, 2), pos=ex),
    lambda: mx.moe_combine(z(8, 64, dtype=F32), pos=ex),
    lambda: mx.moe_combine_backward(x, z(8, 64), pos=ex),
    lambda: mx.moe_combine_backward(z(3, 64), z(8, 64), pos=ex, slots=z(8, dtype=I32)),
    lambda: mx.moe_combine_backward(x, z(8, 64), pos=ex, slots=z(9, dtype=I32)),
]


@pytest.mark.parametrize("i", range(len(WRONG)))
def test_binding_refuses(i):
    with pytest.raises((TypeError, ValueError)) as e:
        WRONG[i]()
    assert "ROCm" not in str(e.value)          # its own check, not the device's


@pytest.mark.parametrize("good", [
    lambda: mx.mx_rmsnorm(x, z(64), residual=x, axis=3, checkpoint=True),
    lambda: mx.mx_rmsnorm_backward(x, z(4, dtype=F32), z(64), h=x, dres=x),
    lambda: mx.moe_route(lg, 2, bias=z(8, dtype=F32), want_scores=True),
    lambda: mx.moe_route_backward(z(4, 2, dtype=F32), lg, ex),
    lambda: mx.moe_sort(ex, 8),
    lambda: mx.moe_gather(x, z(8, dtype=I32), 2),
    lambda: mx.moe_combine(z(8, 64), weights=z(4, 2, dtype=F32), pos=ex),
    lambda: mx.moe_combine(z(4, 2, 64)),
    lambda: mx.moe_combine_backward(x, z(8, 64), pos=ex, slots=z(8, dtype=I32)),
], ids=["norm", "norm_back", "route", "route_back", "sort", "gather", "combine", "combine3", "combine_back"])
def test_binding_wants_a_device(good):
    with pytest.raises(ValueError, match="ROCm"):
        good()
