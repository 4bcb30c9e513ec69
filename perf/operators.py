"""The library's matrix products on block-scaled operands, as workloads.

Four operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and through the library:

  matmul         y[M][N] = A B^T, A [M][K] and B [N][K] MXFP8: a dense layer's
                 forward product or input gradient
  matmul_grouped the same for G experts stacked along rows: group g's rows of A
                 by the expert's own B_g [N][K]
  wgrad_grouped  dW_g[N][K] = sum over the group's rows m of dY[m][n] X[m][k],
                 from the transposed (column-wise) MXFP8 casts of dY and X
  matvec         y[T][N] = x W^T, x bf16 [T][K], W [N][K] NVFP4 (4-bit elements,
                 an E4M3 scale per 16, an fp32 tensor scale): decoding
  matvec_experts y[t][j] = x[t] W_e^T with e = experts[t][j]: decoding through
                 the experts a router picked; an index outside 0 .. G - 1 (a
                 padded slot, an expert on another device) gives a row of zeros

matmul and matmul_grouped are one operator (a dense product is one group).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    # rows: all groups' rows; step: rows per group are multiples of it (but
    # one group's, which takes the remainder); split: seed of the group sizes;
    # a, b: element formats of the two operands; tiled: the scale layout
    return [
        # the up projection [gate | linear] of an MoE layer of 8 experts over
        # 16384 tokens, expert sizes padded to 16, scales in MFMA tiles
        dict(name="experts_up", op="matmul_grouped", groups=8, rows=16384, step=16, split=8,
             n=4096, k=7168, a="e4m3", b="e4m3", tiled=True, out="bf16"),
        # the same layer's input gradient: E5M2 gradients, expert sizes as the
        # router left them, compact scales
        dict(name="experts_dgrad", op="matmul_grouped", groups=8, rows=16384, step=1, split=8,
             n=7168, k=4096, a="e5m2", b="e4m3", tiled=False, out="bf16"),
        # decoding a small batch through MXFP8 experts: a few rows each, some
        # experts without any
        dict(name="experts_small", op="matmul_grouped", groups=16, rows=64, step=1, split=3,
             n=4096, k=2048, a="e4m3", b="e4m3", tiled=False, out="bf16"),
        # a dense layer
        dict(name="dense", op="matmul", m=8192, n=8192, k=8192, a="e4m3", b="e4m3", tiled=True,
             out="bf16"),
        # a small odd product: every edge partial, rows at any byte
        dict(name="dense_odd", op="matmul", m=200, n=333, k=1111, a="e4m3", b="e4m3", tiled=False,
             out="f32"),
        # the up projection's weight gradients, expert sizes padded to 16
        dict(name="experts_wgrad", op="wgrad_grouped", groups=8, rows=16384, step=16, split=8,
             n=4096, k=7168, a="e5m2", b="e4m3", tiled=True, out="f32"),
        # weight gradients of a smaller layer with unpadded expert sizes: the
        # transposed rows start at any byte
        dict(name="experts_wgrad_ragged", op="wgrad_grouped", groups=8, rows=8192, step=1, split=5,
             n=2048, k=5120, a="e4m3", b="e4m3", tiled=False, out="bf16"),
        # one token through a projection
        dict(name="token", op="matvec", t=1, n=14336, k=4096, out="bf16"),
        # a batch of tokens through a large matrix
        dict(name="batch", op="matvec", t=16, n=16384, k=16384, out="bf16"),
        # odd sizes: half-filled last bytes, partial blocks, rows at any byte
        dict(name="batch_odd", op="matvec", t=5, n=1001, k=4095, out="f32"),
        # one token through two of eight experts
        dict(name="token_experts", op="matvec_experts", t=1, top=2, groups=8, n=5120, k=4096,
             pad=0, out="bf16"),
        # a padded batch through four of sixteen experts
        dict(name="batch_experts", op="matvec_experts", t=32, top=4, groups=16, n=4096, k=2048,
             pad=3, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm: as often a
    multiple of 128 or of 16 as any number."""
    n, step = _log(rng, lo, hi), rng.choice((1, 1, 16, 128))
    return max(lo, n // step * step)


def draw(rng):
    op = rng.choice(("matmul", "matmul_grouped", "wgrad_grouped", "matvec", "matvec_experts"))
    out = rng.choice(("bf16", "f32"))
    if op == "matvec":
        t, n = rng.choice((1, 2, _log(rng, 1, 64))), _dim(rng, 64, 16384)
        return dict(op=op, t=t, n=n, k=_dim(rng, 64, 16384), out=out)
    if op == "matvec_experts":
        g = rng.choice((4, 8, 16, 32))
        t, k = _log(rng, 1, 64), _dim(rng, 64, 8192)
        # no more weights than a listed case's 2^28
        return dict(op=op, t=t, top=rng.randint(1, 4), groups=g,
                    n=_dim(rng, 64, max(64, min(8192, 2 ** 28 // (g * k)))), k=k,
                    pad=rng.randint(0, t - 1) if t > 1 else 0, out=out)
    fmt = dict(a=rng.choice(("e4m3", "e5m2")), b=rng.choice(("e4m3", "e4m3", "e5m2")),
               tiled=rng.random() < 0.5, out=out)
    if op == "matmul":
        return dict(op=op, m=_dim(rng, 16, 8192), n=_dim(rng, 64, 8192), k=_dim(rng, 64, 8192),
                    **fmt)
    g, rows, k = rng.choice((2, 4, 8, 8, 16, 32)), _log(rng, 16, 16384), _dim(rng, 64, 7168)
    # no more weights than those of 8 experts of 4096 x 7168
    return dict(op=op, groups=g, rows=rows, step=rng.choice((1, 16, 128)),
                split=rng.randint(1, 1000),
                n=_dim(rng, 64, max(64, min(4096, 8 * 4096 * 7168 // (g * k)))), k=k, **fmt)


def group_rows(case):
    """Rows of each group: uneven shares, rounded down to `step`; the largest
    group takes what is left over."""
    r = np.random.default_rng(case["split"])
    share = r.dirichlet(np.ones(case["groups"]))
    rows = [int(v) // case["step"] * case["step"] for v in share * case["rows"]]
    rows[int(np.argmax(share))] += case["rows"] - sum(rows)
    return rows


def work(case):
    op, out = case["op"], 2 if case["out"] == "bf16" else 4

    def mx(rows, cols):
        return rows * cols + rows * -(-cols // 32)

    def nv(rows, cols):
        return rows * (-(-cols // 2) + -(-cols // 16))

    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return dict(bytes=mx(m, k) + mx(n, k) + out * m * n, flops=2 * m * n * k)
    if op == "matmul_grouped":
        m, n, k = case["rows"], case["n"], case["k"]
        used = sum(1 for r in group_rows(case) if r)
        return dict(bytes=mx(m, k) + used * mx(n, k) + out * m * n, flops=2 * m * n * k)
    if op == "wgrad_grouped":
        m, n, k, g = case["rows"], case["n"], case["k"], case["groups"]
        return dict(bytes=sum(mx(n, r) + mx(k, r) for r in group_rows(case)) + out * g * n * k,
                    flops=2 * m * n * k)
    t, n, k = case["t"], case["n"], case["k"]
    if op == "matvec":
        return dict(bytes=nv(n, k) + 2 * t * k + out * t * n, flops=2 * t * n * k)
    live, slots = t - case["pad"], t * case["top"]
    used = min(case["groups"], live * case["top"])
    return dict(bytes=used * nv(n, k) + 2 * live * k + 4 * slots + out * slots * n,
                flops=2 * live * case["top"] * n * k)


# ---- inputs -----------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _values(g, rows, cols):
    """Activations, weights or gradients: normal values whose rows differ in
    magnitude."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    return x * torch.exp2(torch.randint(-3, 3, (rows, 1), generator=g, device=DEV).float())


def _mxfp8(x, fmt):
    """MXFP8 of x along its rows: codes [R][C] and scale bytes [R][ceil(C/32)]."""
    R, C = x.shape
    nb = -(-C // 32)
    p = torch.nn.functional.pad(x, (0, nb * 32 - C)).view(R, nb, 32)
    emax, top, dtype = ((8, 448.0, torch.float8_e4m3fn) if fmt == "e4m3" else
                        (15, 57344.0, torch.float8_e5m2))
    amax = p.abs().amax(-1, keepdim=True)
    byte = (torch.floor(torch.log2(amax.clamp_min(1e-37))) - emax + 127).clamp(0, 254)
    q = (p * torch.exp2(127 - byte)).clamp(-top, top).to(dtype).view(torch.uint8)
    return q.view(R, nb * 32)[:, :C].contiguous(), byte.view(R, nb).to(torch.uint8)


def _tile(s):
    """Scale bytes [R][C] in the tile layout: 32-row x 8-block tiles of 256
    bytes, tile (rt, bt) at (bt * RT + rt) * 256, word L of a tile holding in
    byte j the scale of row L % 32 and block 2j + L / 32."""
    R, C = s.shape
    RT, CT = -(-R // 32), -(-C // 8)
    s = torch.nn.functional.pad(s, (0, CT * 8 - C, 0, RT * 32 - R))
    return s.view(RT, 32, CT, 4, 2).permute(2, 0, 4, 1, 3).reshape(-1)


def _operand(x, fmt, tiled):
    q, s = _mxfp8(x, fmt)
    return q.view(-1), _tile(s) if tiled else s.reshape(-1)


def _groups_of(parts, sizes, like):
    """The groups' tensors one after the other (an empty group has none)."""
    live = [p for p, r in zip(parts, sizes) if r]
    return torch.cat([p[0] for p in live]), torch.cat([p[1] for p in live])


def _nvfp4(x):
    """NVFP4 of x along its rows: packed codes [R][ceil(C/2)], E4M3 scale bytes
    [R][ceil(C/16)] and the tensor scale."""
    R, C = x.shape
    nb = -(-C // 16)
    p = torch.nn.functional.pad(x, (0, nb * 16 - C)).view(R, nb, 16)
    sg = (x.abs().amax() / 2688.0).view(1)
    s = (p.abs().amax(-1) / 6.0 / sg).clamp(max=448.0).to(torch.float8_e4m3fn)
    div = s.float() * sg
    p = p * torch.where(div > 0, 1.0 / div, torch.zeros_like(div)).unsqueeze(-1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(p.abs(), edges).to(torch.uint8) + 8 * (p < 0).to(torch.uint8)
    code = code.view(R, nb * 16)
    code[:, C:] = 0
    packed = code[:, 0::2] + 16 * code[:, 1::2]
    return packed[:, :-(-C // 2)].contiguous(), s.view(torch.uint8), sg


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    odtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    st = dict(case=case)
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        st["qa"], st["sa"] = _operand(_values(g, m, k), case["a"], case["tiled"])
        st["qb"], st["sb"] = _operand(_values(g, n, k), case["b"], case["tiled"])
        st["qa"], st["qb"] = st["qa"].view(m, k), st["qb"].view(n, k)
        st["out"] = torch.empty(m, n, dtype=odtype, device=DEV)
    elif op in ("matmul_grouped", "wgrad_grouped"):
        n, k, m, rows = case["n"], case["k"], case["rows"], group_rows(case)
        st["rows"] = rows
        if op == "matmul_grouped":
            a = [_operand(_values(g, r, k), case["a"], case["tiled"]) if r else None for r in rows]
            b = [_operand(_values(g, n, k), case["b"], case["tiled"]) for _ in rows]
            st["qa"], st["sa"] = _groups_of(a, rows, m)
            st["qb"], st["sb"] = _groups_of(b, [1] * len(rows), m)
            st["qa"] = st["qa"].view(m, k)
            st["out"] = torch.empty(m, n, dtype=odtype, device=DEV)
        else:
            a = [_operand(_values(g, n, r), case["a"], case["tiled"]) if r else None for r in rows]
            b = [_operand(_values(g, k, r), case["b"], case["tiled"]) if r else None for r in rows]
            st["qa"], st["sa"] = _groups_of(a, rows, m)
            st["qb"], st["sb"] = _groups_of(b, rows, m)
            st["out"] = torch.empty(len(rows), n, k, dtype=odtype, device=DEV)
    else:
        t, n, k = case["t"], case["n"], case["k"]
        G = case.get("groups", 1)
        st["x"] = _values(g, t, k).to(torch.bfloat16)
        w = [_nvfp4(_values(g, n, k)) for _ in range(G)]
        st["qw"], st["sw"], st["sg"] = (torch.cat([p[i] for p in w]) for i in range(3))
        if op == "matvec":
            st["out"] = torch.empty(t, n, dtype=odtype, device=DEV)
        else:
            top = case["top"]
            # distinct experts per token; the padded slots at the end hold -1;
            # the first tokens go through the experts in turn, so that as many
            # are used as the batch can reach
            order = torch.rand(t, G, generator=g, device=DEV).argsort(1)[:, :top]
            turn = (torch.arange(t * top, device=DEV) + int(seed) % G) % G
            e = torch.where((torch.arange(t, device=DEV) * top < G).unsqueeze(1) |
                            torch.tensor(top >= G, device=DEV), turn.view(t, top), order)
            live = t - case["pad"]
            e = torch.where((torch.arange(t, device=DEV) < live).unsqueeze(1), e,
                            torch.full_like(e, -1))
            st["experts"] = e.to(torch.int32).contiguous()
            st["out"] = torch.empty(t, top, n, dtype=odtype, device=DEV)
    return st


# ---- the plain form ---------------------------------------------------------

def _untile(flat, R, C):
    RT, CT = -(-R // 32), -(-C // 8)
    s = flat.view(CT, RT, 2, 32, 4).permute(1, 3, 0, 4, 2).reshape(RT * 32, CT * 8)
    return s[:R, :C]


def _scale_bytes(R, C, tiled):
    nb = -(-C // 32)
    return -(-R // 32) * -(-nb // 8) * 256 if tiled else R * nb


def _mx_values(q, s, R, C, fmt, tiled):
    """The fp32 values of an MXFP8 operand [R][C]."""
    nb = -(-C // 32)
    s = _untile(s, R, nb) if tiled else s.view(R, nb)
    scale = torch.where(s == 255, torch.full((), float("nan"), device=DEV),
                        torch.exp2(s.float() - 127))
    dtype = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    v = q.reshape(R, C).view(dtype).float()
    return v * scale.repeat_interleave(32, 1)[:, :C]


def _nv_values(q, s, sg, K):
    """The fp32 values of an NVFP4 matrix [N][K]."""
    mag = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6.], device=DEV)
    table = torch.cat([mag, -mag])
    code = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1)[:, :K]
    scale = s.view(torch.float8_e4m3fn).float().repeat_interleave(16, 1)[:, :K]
    return table[code.int()] * scale * sg


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    dt = st["out"].dtype
    if op == "matmul":
        a = _mx_values(st["qa"], st["sa"], case["m"], case["k"], case["a"], case["tiled"])
        b = _mx_values(st["qb"], st["sb"], case["n"], case["k"], case["b"], case["tiled"])
        return (a @ b.t()).to(dt)
    if op in ("matmul_grouped", "wgrad_grouped"):
        n, k, tiled, ys = case["n"], case["k"], case["tiled"], []
        qa, qb, sa, sb = (st[i].view(-1) for i in ("qa", "qb", "sa", "sb"))
        for r in st["rows"]:
            (ra, ca), (rb, cb) = ((r, k), (n, k)) if op == "matmul_grouped" else ((n, r), (k, r))
            if r == 0:
                if op == "matmul_grouped":
                    qb, sb = qb[rb * cb:], sb[_scale_bytes(rb, cb, tiled):]
                else:
                    ys.append(torch.zeros(n, k, device=DEV))
                continue
            na, nb = _scale_bytes(ra, ca, tiled), _scale_bytes(rb, cb, tiled)
            a = _mx_values(qa[:ra * ca], sa[:na], ra, ca, case["a"], tiled)
            b = _mx_values(qb[:rb * cb], sb[:nb], rb, cb, case["b"], tiled)
            ys.append(a @ b.t())
            qa, sa, qb, sb = qa[ra * ca:], sa[na:], qb[rb * cb:], sb[nb:]
        y = torch.cat(ys) if op == "matmul_grouped" else torch.stack(ys)
        return y.to(dt)
    n, k, x = case["n"], case["k"], st["x"].float()
    if op == "matvec":
        return (x @ _nv_values(st["qw"], st["sw"], st["sg"], k).t()).to(dt)
    e = st["experts"]
    y = torch.zeros(case["t"], case["top"], n, device=DEV)
    for g in range(case["groups"]):
        w = _nv_values(st["qw"][g * n:(g + 1) * n], st["sw"][g * n:(g + 1) * n], st["sg"][g], k)
        y = torch.where((e == g).unsqueeze(-1), (x @ w.t()).unsqueeze(1), y)
    return y.to(dt)


def run(st):
    if not own:
        return _plain(st)
    import block_scaled_precision_bf16_amd as mx
    case, op = st["case"], st["case"]["op"]
    flags = mx.OUT_F32 if case["out"] == "f32" else 0
    if op == "matvec":
        return mx.nvfp4_matvec(st["x"], st["qw"], st["sw"], st["sg"], flags=flags, out=st["out"])
    if op == "matvec_experts":
        return mx.nvfp4_matvec_experts(st["x"], st["experts"], st["qw"], st["sw"], st["sg"],
                                       flags=flags, out=st["out"])
    flags |= (mx.A_E5M2 if case["a"] == "e5m2" else 0) | (mx.B_E5M2 if case["b"] == "e5m2" else 0) \
        | (mx.SCALE_TILED if case["tiled"] else 0)
    args = (st["qa"], st["sa"], st["qb"], st["sb"])
    if op == "matmul":
        return mx.mx_matmul(*args, flags=flags, out=st["out"])
    if op == "matmul_grouped":
        return mx.mx_matmul_grouped(*args, st["rows"], flags=flags, out=st["out"])
    return mx.mx_matmul_wgrad_grouped(*args, st["rows"], flags=flags, out=st["out"])


# ---- the definition in 64 bits ----------------------------------------------

def _fp8_table(ebits, mbits):
    """Value of every code of an 8-bit float with these fields (bias
    2^(ebits-1) - 1); the codes the formats reserve are NaN (or infinite)."""
    bias, vals = 2 ** (ebits - 1) - 1, []
    for c in range(256):
        e, m = (c >> mbits) & (2 ** ebits - 1), c & (2 ** mbits - 1)
        v = math.ldexp(m, 1 - bias - mbits) if e == 0 else math.ldexp(2 ** mbits + m, e - bias - mbits)
        if ebits == 4 and c & 127 == 127:
            v = math.nan
        if ebits == 5 and e == 31:
            v = math.inf if m == 0 else math.nan
        vals.append(-v if c & 128 else v)
    return torch.tensor(vals, dtype=torch.float64, device=DEV)


def _exact_operand(q, s, R, C, fmt, tiled):
    nb = -(-C // 32)
    if tiled:
        r, b = torch.arange(R, device=DEV).unsqueeze(1), torch.arange(nb, device=DEV).unsqueeze(0)
        tile = (b // 8) * -(-R // 32) + r // 32
        s = s[tile * 256 + 4 * (r % 32 + 32 * (b % 2)) + (b % 8) // 2]
    else:
        s = s.view(R, nb)
    e = 2.0 ** (torch.arange(256, dtype=torch.float64, device=DEV) - 127)
    e[255] = math.nan
    table = _fp8_table(4, 3) if fmt == "e4m3" else _fp8_table(5, 2)
    col = torch.arange(C, device=DEV) // 32
    return table[q.reshape(R, C).int()] * e[s.int()][:, col]


def _exact_weight(q, s, sg, K):
    mag = [0, 1, 2, 3, 4, 6, 8, 12]
    table = torch.tensor([v / 2 for v in mag] + [-v / 2 for v in mag], dtype=torch.float64, device=DEV)
    col = torch.arange(K, device=DEV)
    code = (q[:, col // 2].int() >> (4 * (col % 2)).int()) & 15
    return table[code] * _fp8_table(4, 3)[s.int()][:, col // 16] * sg.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "matmul":
        a = _exact_operand(st["qa"], st["sa"], case["m"], case["k"], case["a"], case["tiled"])
        b = _exact_operand(st["qb"], st["sb"], case["n"], case["k"], case["b"], case["tiled"])
        return torch.mm(a, b.t())
    if op in ("matmul_grouped", "wgrad_grouped"):
        n, k, tiled, rows = case["n"], case["k"], case["tiled"], st["rows"]
        qa, qb = st["qa"].view(-1), st["qb"].view(-1)
        y = torch.zeros((case["rows"], n) if op == "matmul_grouped" else (len(rows), n, k),
                        dtype=torch.float64, device=DEV)
        a0 = b0 = sa0 = sb0 = r0 = 0
        for g, r in enumerate(rows):
            shape_a, shape_b = ((r, k), (n, k)) if op == "matmul_grouped" else ((n, r), (k, r))
            ea, eb = shape_a[0] * shape_a[1], shape_b[0] * shape_b[1]
            la = _scale_bytes(*shape_a, tiled) if r else 0
            lb = _scale_bytes(*shape_b, tiled) if r or op == "matmul_grouped" else 0
            if r:
                a = _exact_operand(qa[a0:a0 + ea], st["sa"][sa0:sa0 + la], *shape_a, case["a"], tiled)
                b = _exact_operand(qb[b0:b0 + eb], st["sb"][sb0:sb0 + lb], *shape_b, case["b"], tiled)
                p = torch.mm(a, b.t())
                if op == "matmul_grouped":
                    y[r0:r0 + r] = p
                else:
                    y[g] = p
            a0, b0, sa0, sb0, r0 = a0 + ea, b0 + eb, sa0 + la, sb0 + lb, r0 + r
        return y
    n, k, x = case["n"], case["k"], st["x"].double()
    if op == "matvec":
        return torch.mm(x, _exact_weight(st["qw"], st["sw"], st["sg"], k).t())
    y = torch.zeros(case["t"], case["top"], n, dtype=torch.float64, device=DEV)
    chosen = st["experts"].tolist()
    for g in range(case["groups"]):
        slots = [(t, j) for t, row in enumerate(chosen) for j, e in enumerate(row) if e == g]
        if slots:
            w = _exact_weight(st["qw"][g * n:(g + 1) * n], st["sw"][g * n:(g + 1) * n], st["sg"][g], k)
            t, j = (torch.tensor(c, device=DEV) for c in zip(*slots))
            y[t, j] = torch.mm(x[t], w.t())
    return y
