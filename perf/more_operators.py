"""What stands around the library's casts and products in a transformer layer
with experts, as workloads.

Three operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and through the library:

  norm          h = x + residual, its root-mean-square norm y = h rstd w, and
                the MXFP8 casts of y that the next product takes (rows, columns
                or both), with h itself kept in 8 bits on request
  norm_back     the norm's gradients from h, or from the 8-bit h
  route         a router's logits to each token's experts and weights: softmax
                or sigmoid scores, a bias for balance, groups, top-k
  route_back    the gradient of the logits
  dispatch      the tokens' rows stacked by expert, the order that the grouped
                casts and products take
  combine       the experts' rows back to tokens, weighted
  combine_back  its gradients: of the experts' rows and of the weights

dispatch and combine are one operator (to the experts and back).
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E8M0 = torch.float8_e8m0fnu


def listed():
    return [
        # the norm before the up projection of an MoE layer in training: 16384
        # tokens of 7168, casts for the product and for its weight gradient
        # (scales in MFMA tiles), the residual stream kept in 8 bits
        dict(name="norm_train", op="norm", m=16384, k=7168, residual=True, axis=3, fmt="e4m3",
             up=False, tiled=True, ckpt=True, y=False),
        # a chunk of a prompt, forward only
        dict(name="norm_prefill", op="norm", m=2048, k=8192, residual=True, axis=1, fmt="e4m3",
             up=False, tiled=False, ckpt=False, y=False),
        # one token of a decoded batch: bf16 out, as the NVFP4 products take it
        dict(name="norm_token", op="norm", m=1, k=4096, residual=True, axis=0, fmt="e4m3",
             up=False, tiled=False, ckpt=False, y=True),
        # odd sizes: partial blocks, rows at any byte, no residual
        dict(name="norm_odd", op="norm", m=333, k=1111, residual=False, axis=3, fmt="e5m2",
             up=True, tiled=False, ckpt=False, y=True),
        # the backward of the first, from bf16 and with the residual's gradient
        dict(name="norm_back", op="norm_back", m=16384, k=7168, dres=True, ckpt=False),
        # the backward from an 8-bit checkpoint, a shorter batch of uneven rows
        dict(name="norm_back_ckpt", op="norm_back", m=2001, k=5120, dres=True, ckpt=True),
        # training through 256 experts in 8 groups, 8 of them for each token
        dict(name="route_train", op="route", t=16384, e=256, top=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, pair=True, renorm=True, logits="f32", masked=0.0, scores=False),
        # a decoded batch, 4 of 64 experts, some experts masked
        dict(name="route_batch", op="route", t=32, e=64, top=4, score="softmax", bias=False,
             groups=1, top_groups=1, pair=False, renorm=True, logits="bf16", masked=0.3,
             scores=False),
        # a router's gradient, with that of a balance loss on the scores
        dict(name="route_back", op="route_back", t=16384, e=64, top=8, score="softmax",
             renorm=True, logits="f32", masked=0.0, scores=True),
        # 4096 tokens to 4 of 8 experts: 16384 rows, expert sizes padded to 16
        dict(name="dispatch", op="dispatch", t=4096, top=4, e=8, align=16, k=7168, pad=0),
        # the products of a decoded batch back to its tokens
        dict(name="combine_batch", op="combine", t=32, top=8, e=256, align=1, k=4096, pad=3,
             sorted=False, weights=True),
        # the backward of 4096 tokens' way back from their experts
        dict(name="combine_back", op="combine_back", t=4096, top=4, e=8, align=16, k=7168, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm: as often a
    multiple of 128 or of 8 as any number."""
    n, step = _log(rng, lo, hi), rng.choice((1, 8, 8, 128))
    return max(lo, n // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_back", "route", "route_back", "dispatch", "combine",
                     "combine_back"))
    if op in ("norm", "norm_back"):
        k = _dim(rng, 32, 16384)
        # no more elements than the listed 16384 x 7168
        m = _dim(rng, 1, min(16384, 16384 * 7168 // k))
        if op == "norm_back":
            return dict(op=op, m=m, k=k, dres=rng.random() < 0.7, ckpt=rng.random() < 0.5)
        axis = rng.choice((0, 1, 2, 3, 3))
        return dict(op=op, m=m, k=k, residual=rng.random() < 0.7, axis=axis,
                    fmt=rng.choice(("e4m3", "e4m3", "e5m2")), up=rng.random() < 0.3,
                    tiled=rng.random() < 0.5, ckpt=rng.random() < 0.3,
                    y=axis == 0 or rng.random() < 0.2)
    if op in ("route", "route_back"):
        e = rng.choice((4, 8, 16, 40, 64, 128, 160, 256))
        t, top = _log(rng, 1, min(65536, 2 ** 22 // e)), rng.randint(1, min(e, 10))
        score, logits = rng.choice(("softmax", "sigmoid")), rng.choice(("f32", "bf16"))
        masked = rng.choice((0.0, 0.0, 0.3))
        c = dict(op=op, t=t, e=e, top=top, score=score, renorm=rng.random() < 0.6, logits=logits,
                 masked=masked, scores=rng.random() < 0.4)
        if op == "route":
            groups = rng.choice([g for g in (1, 1, 2, 4, 8) if e % g == 0 and e // g >= 2])
            c.update(bias=rng.random() < 0.5, groups=groups, top_groups=rng.randint(1, groups),
                     pair=rng.random() < 0.5)
        return c
    e = rng.choice((4, 8, 16, 64, 256))
    top, k = rng.randint(1, min(8, e)), _dim(rng, 64, 8192)
    t = _log(rng, 1, max(1, 16384 * 7168 // (top * k)))
    t = min(t, 65536 // top)
    c = dict(op=op, t=t, top=top, e=e, align=rng.choice((1, 16, 32)), k=k,
             pad=rng.randint(0, t // 4))
    if op == "combine":
        c.update(sorted=rng.random() < 0.7, weights=rng.random() < 0.8)
    return c


def _capacity(case):
    """Rows that hold every expert's slots, each expert's padded to `align`."""
    slots = case["t"] * case["top"]
    return slots + min(case["e"], slots) * (case["align"] - 1)


def work(case):
    op = case["op"]
    if op == "norm":
        m, k, a = case["m"], case["k"], case["axis"]
        n, row, col = m * k, m * k + m * -(-k // 32), m * k + k * -(-m // 32)
        return dict(bytes=2 * n + (4 * n if case["residual"] else 0) + (2 * n if case["y"] else 0) +
                    (row if a & 1 else 0) + (col if a & 2 else 0) + (row if case["ckpt"] else 0) +
                    4 * m + 2 * k, flops=5 * n)
    if op == "norm_back":
        m, k = case["m"], case["k"]
        n = m * k
        return dict(bytes=2 * n + (n + m * -(-k // 32) if case["ckpt"] else 2 * n) +
                    (2 * n if case["dres"] else 0) + 2 * n + 4 * m + 6 * k, flops=10 * n)
    if op in ("route", "route_back"):
        t, e, size = case["t"], case["e"], 4 if case["logits"] == "f32" else 2
        scores = 4 * t * e if case["scores"] else 0
        if op == "route":
            return dict(bytes=size * t * e + 8 * t * case["top"] + scores +
                        (4 * e if case["bias"] else 0), flops=10 * t * e)
        return dict(bytes=2 * size * t * e + 8 * t * case["top"] + scores, flops=10 * t * e)
    t, top, k, live = case["t"], case["top"], case["k"], case["t"] - case["pad"]
    slots = live * top
    if op == "dispatch":
        return dict(bytes=4 * t * top + 2 * live * k + 2 * _capacity(case) * k + 4 * t * top +
                    4 * _capacity(case) + 4 * case["e"], flops=0)
    if op == "combine":
        read = slots if case["sorted"] else t * top
        return dict(bytes=2 * read * k + 2 * t * k + (4 * t * top if case["sorted"] else 0) +
                    (4 * t * top if case["weights"] else 0), flops=2 * slots * k)
    return dict(bytes=2 * live * k + 2 * slots * k + 2 * _capacity(case) * k + 12 * t * top +
                4 * _capacity(case), flops=3 * slots * k)


# ---- inputs -----------------------------------------------------------------

def _values(g, rows, cols):
    """Activations or gradients: normal values whose rows differ in magnitude."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    return (x * torch.exp2(torch.randint(-3, 3, (rows, 1), generator=g, device=DEV).float())).to(BF16)


def _chosen(g, case):
    """Distinct experts for each token; the padded tokens at the end have none."""
    t = case["t"]
    e = torch.rand(t, case["e"], generator=g, device=DEV).argsort(1)[:, :case["top"]]
    live = torch.arange(t, device=DEV) < t - case.get("pad", 0)
    return torch.where(live.unsqueeze(1), e, torch.full_like(e, -1)).to(torch.int32).contiguous()


def _sorted(experts, n, align, rows):
    """Stable order by expert, each expert's rows from a multiple of `align`:
    rows of each expert, each slot's row and each row's slot (-1: none)."""
    flat = experts.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < n), flat, torch.full_like(flat, n))
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=n + 1)
    padded = (counts + align - 1) // align * align
    first, start = counts.cumsum(0) - counts, padded.cumsum(0) - padded
    by = key[order]
    row = torch.arange(flat.numel(), device=DEV) - first[by] + start[by]
    live = by < n
    pos = torch.full_like(flat, -1)
    pos[order] = torch.where(live, row, torch.full_like(row, -1))
    slots = torch.full((rows + 1,), -1, dtype=torch.long, device=DEV)
    slots[torch.where(live, row, torch.full_like(row, rows))] = order
    slots[rows] = -1
    return (counts[:n].to(torch.int32), pos.view(experts.shape).to(torch.int32),
            slots[:rows].to(torch.int32))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, st = case["op"], dict(case=case)
    if op in ("norm", "norm_back"):
        m, k = case["m"], case["k"]
        st["w"] = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(BF16)
        if op == "norm":
            st["x"] = _values(g, m, k)
            st["res"] = _values(g, m, k) if case["residual"] else None
            return st
        h = _values(g, m, k)
        st["rstd"] = torch.rsqrt(h.float().square().mean(1) + 1e-6)
        st["h"] = h
        if case["ckpt"]:
            st["h"] = None
            st["q_h"], st["s_h"] = _mxfp8(h, "e4m3", True)
        st["dy"] = _values(g, m, k)
        st["dres"] = _values(g, m, k) if case["dres"] else None
        return st
    if op in ("route", "route_back"):
        t, e = case["t"], case["e"]
        x = 1.5 * torch.randn(t, e, generator=g, device=DEV)
        if case["masked"]:
            off = torch.rand(t, e, generator=g, device=DEV) < case["masked"]
            off[t // 2] = True     # a token whose mask leaves nothing
            x = x.masked_fill(off, float("-inf"))
        st["logits"] = x.to(F32 if case["logits"] == "f32" else BF16)
        if op == "route":
            st["bias"] = 0.1 * torch.randn(e, generator=g, device=DEV) if case["bias"] else None
            return st
        key = st["logits"].float()
        best, order = torch.sort(key, dim=1, descending=True, stable=True)
        top = case["top"]
        st["experts"] = torch.where(best[:, :top] > float("-inf"), order[:, :top],
                                    torch.full_like(order[:, :top], -1)).to(torch.int32).contiguous()
        st["dweights"] = torch.randn(t, top, generator=g, device=DEV)
        st["dscores"] = 0.1 * torch.randn(t, e, generator=g, device=DEV) if case["scores"] else None
        return st
    t, top, k = case["t"], case["top"], case["k"]
    st["experts"] = _chosen(g, case)
    if op == "dispatch":
        st["x"] = _values(g, t, k)
        return st
    rows = _capacity(case)
    st["weights"] = torch.rand(t, top, generator=g, device=DEV)
    if op == "combine":
        if not case["weights"]:
            st["weights"] = None
        if case["sorted"]:
            st["pos"] = _sorted(st["experts"], case["e"], case["align"], rows)[1]
            st["y"] = _values(g, rows, k)
        else:
            st["pos"] = None
            y = _values(g, t * top, k)
            st["y"] = y.masked_fill(st["experts"].view(-1, 1) < 0, 0.0).view(t, top, k)
        return st
    _, st["pos"], st["slots"] = _sorted(st["experts"], case["e"], case["align"], rows)
    st["y"] = _values(g, rows, k)
    st["dout"] = _values(g, t, k)
    return st


# ---- the plain form ---------------------------------------------------------

def _tile(s):
    """Scale bytes [R][C] in the tile layout: 32-row x 8-block tiles of 256
    bytes, tile (rt, bt) at (bt * RT + rt) * 256, word L of a tile holding in
    byte j the scale of row L % 32 and block 2j + L / 32."""
    R, C = s.shape
    RT, CT = -(-R // 32), -(-C // 8)
    s = torch.nn.functional.pad(s, (0, CT * 8 - C, 0, RT * 32 - R))
    return s.view(RT, 32, CT, 4, 2).permute(2, 0, 4, 1, 3).reshape(-1)


def _mxfp8(x, fmt, up):
    """MXFP8 of bf16 x along its rows: elements [R][C] (float8) and scale bytes
    [R][ceil(C/32)]."""
    R, C = x.shape
    nb = -(-C // 32)
    p = torch.nn.functional.pad(x.float(), (0, nb * 32 - C)).view(R, nb, 32)
    emax, top, dtype = ((8, 448.0, torch.float8_e4m3fn) if fmt == "e4m3" else
                        (15, 57344.0, torch.float8_e5m2))
    mant, e = torch.frexp(p.abs().amax(-1, keepdim=True))
    byte = e - 1 - emax + 127 + ((mant > 0.875).int() if up else 0)
    byte = torch.where(mant == 0, torch.zeros_like(byte), byte).clamp(0, 254)
    q = torch.ldexp(p, 127 - byte).clamp(-top, top).to(dtype).view(R, nb * 32)
    return q[:, :C].contiguous(), byte.view(R, nb).to(torch.uint8)


def _cast(y, case):
    """The norm's MXFP8 outputs along one direction, scales in the case's layout."""
    q, s = _mxfp8(y, case["fmt"], case["up"])
    return q, (_tile(s) if case["tiled"] else s).view(E8M0)


def _plain_norm(st):
    case, x = st["case"], st["x"]
    h = x if st["res"] is None else (x.float() + st["res"].float()).to(BF16)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + 1e-6)
    y = (hf * rstd.unsqueeze(1) * st["w"].float()).to(BF16)
    o = dict(rstd=rstd)
    if st["res"] is not None:
        o["h"] = h
    if case["y"]:
        o["y"] = y
    if case["axis"] & 1:
        o["q_row"], o["s_row"] = _cast(y, case)
    if case["axis"] & 2:
        o["q_col"], o["s_col"] = _cast(y.t(), case)
    if case["ckpt"]:
        o["q_h"], s = _mxfp8(h, "e4m3", True)
        o["s_h"] = s.view(E8M0)
    return o


def _plain_norm_back(st):
    case = st["case"]
    if case["ckpt"]:
        scale = torch.exp2(st["s_h"].float() - 127).repeat_interleave(32, 1)[:, :case["k"]]
        h = st["q_h"].float() * scale
    else:
        h = st["h"].float()
    dy, rstd = st["dy"].float(), st["rstd"].unsqueeze(1)
    xhat, gw = h * rstd, dy * st["w"].float()
    dh = rstd * (gw - xhat * (gw * xhat).mean(1, keepdim=True))
    if st["dres"] is not None:
        dh = dh + st["dres"].float()
    return dict(dh=dh.to(BF16), dweight=(dy * xhat).sum(0))


def _scores(logits, kind, dtype):
    """Softmax or sigmoid scores; those of masked experts (-inf) are 0."""
    x = logits.to(dtype)
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    x = torch.exp(x - x.amax(1, keepdim=True).clamp_min(-1e30))
    s = x.sum(1, keepdim=True)
    return x / torch.where(s > 0, s, torch.ones_like(s))


def _plain_route(st):
    case, x = st["case"], st["logits"]
    t, e = x.shape
    p, low = _scores(x, case["score"], F32), float("-inf")
    # selection: without a bias, and where no scores are added, by the logits
    # themselves; otherwise by 64-bit scores
    if st["bias"] is None and not (case["groups"] > 1 and case["pair"]):
        key = x.double()
    else:
        key = _scores(x, case["score"], F64)
        if st["bias"] is not None:
            key = key + st["bias"].double()
        key = key.masked_fill(x == low, low)
    if case["groups"] > 1:
        g = case["groups"]
        best = torch.sort(key.view(t, g, e // g), dim=2, descending=True).values
        score = best[..., 0]
        if case["pair"]:
            score = score + torch.where(best[..., 1] > low, best[..., 1], torch.zeros_like(score))
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros(t, g, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        key = key.masked_fill(~keep.repeat_interleave(e // g, 1), low)
    best, order = torch.sort(key, dim=1, descending=True, stable=True)
    best, order = best[:, :case["top"]], order[:, :case["top"]]
    w = torch.where(best > low, p.gather(1, order), torch.zeros_like(best, dtype=F32))
    if case["renorm"]:
        s = w.sum(1, keepdim=True)
        w = w / torch.where(s > 0, s, torch.ones_like(s))
    o = dict(experts=torch.where(best > low, order, torch.full_like(order, -1)).to(torch.int32),
             weights=2.5 * w)
    if case["scores"]:
        o["scores"] = p
    return o


def _plain_route_back(st):
    case, x = st["case"], st["logits"]
    p, ex, dw = _scores(x, case["score"], F32), st["experts"].long(), st["dweights"]
    live, at = ex >= 0, ex.clamp_min(0)
    ps = torch.where(live, p.gather(1, at), torch.zeros_like(dw))
    d = torch.where(live, 2.5 * dw, torch.zeros_like(dw))
    if case["renorm"]:
        s = ps.sum(1, keepdim=True)
        s = torch.where(s > 0, s, torch.ones_like(s))
        d = (d - (d * ps).sum(1, keepdim=True) / s) / s
        d = torch.where(live, d, torch.zeros_like(d))
    dp = torch.zeros_like(p).scatter_add_(1, at, d)
    if st["dscores"] is not None:
        dp = dp + st["dscores"]
    if case["score"] == "sigmoid":
        return (dp * p * (1 - p)).to(x.dtype)
    return (p * (dp - (dp * p).sum(1, keepdim=True))).to(x.dtype)


def _plain_dispatch(st):
    case, rows = st["case"], _capacity(st["case"])
    counts, pos, slots = _sorted(st["experts"], case["e"], case["align"], rows)
    x = st["x"][slots.clamp_min(0).long() // case["top"]]
    return dict(counts=counts, pos=pos, slots=slots, x=x.masked_fill(slots.unsqueeze(1) < 0, 0.0))


def _rows_of(st):
    """The slots' rows [T][top][K] in 32 bits (0 where a slot has none)."""
    if st["pos"] is None:
        return st["y"].float()
    y = st["y"][st["pos"].clamp_min(0).long()].float()
    return y.masked_fill(st["pos"].unsqueeze(2) < 0, 0.0)


def _plain_combine(st):
    y = _rows_of(st)
    if st["weights"] is not None:
        y = y * st["weights"].unsqueeze(2)
    return y.sum(1).to(BF16)


def _plain_combine_back(st):
    case, slots = st["case"], st["slots"].clamp_min(0).long()
    dy = st["dout"][slots // case["top"]].float() * st["weights"].view(-1, 1)[slots]
    dy = dy.masked_fill(st["slots"].unsqueeze(1) < 0, 0.0)
    return dict(dy=dy.to(BF16), dweights=(_rows_of(st) * st["dout"].float().unsqueeze(1)).sum(2))


def _own(st):
    import block_scaled_precision_bf16_amd as mx
    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        axis = case["axis"]
        if axis:
            axis |= (mx.ELEM_E5M2 if case["fmt"] == "e5m2" else 0) | \
                (mx.SCALE_ROUND_UP if case["up"] else 0) | (mx.SCALE_TILED if case["tiled"] else 0)
        r = mx.mx_rmsnorm(st["x"], st["w"], residual=st["res"], eps=1e-6, axis=axis,
                          want_y=case["y"], checkpoint=case["ckpt"])
        o, f8 = dict(rstd=r["rstd"]), torch.float8_e5m2 if case["fmt"] == "e5m2" else torch.float8_e4m3fn
        if st["res"] is not None:
            o["h"] = r["h"]
        if case["y"]:
            o["y"] = r["y"]
        if axis & 1:
            o["q_row"], o["s_row"] = r["q_row"].view(f8), r["s_row"].view(E8M0)
        if axis & 2:
            o["q_col"], o["s_col"] = r["q_col"].view(f8), r["s_col"].view(E8M0)
        if case["ckpt"]:
            o["q_h"], o["s_h"] = r["q_h"].view(torch.float8_e4m3fn), r["s_h"].view(E8M0)
        return o
    if op == "norm_back":
        ckpt = dict(q_h=st["q_h"].view(torch.uint8), s_h=st["s_h"]) if case["ckpt"] else dict(h=st["h"])
        r = mx.mx_rmsnorm_backward(st["dy"], st["rstd"], st["w"], dres=st["dres"], **ckpt)
        return dict(dh=r["dh"], dweight=r["dweight"])
    if op in ("route", "route_back"):
        flags = (mx.ROUTE_SIGMOID if case["score"] == "sigmoid" else 0) | \
            (mx.ROUTE_RENORM if case["renorm"] else 0)
        if op == "route_back":
            return mx.moe_route_backward(st["dweights"], st["logits"], st["experts"], flags=flags,
                                         scale=2.5, dscores=st["dscores"])
        r = mx.moe_route(st["logits"], case["top"], bias=st["bias"], scale=2.5,
                         flags=flags | (mx.ROUTE_GROUP_PAIR if case["pair"] else 0),
                         groups=case["groups"], top_groups=case["top_groups"],
                         want_scores=case["scores"])
        return {n: v for n, v in r.items() if v is not None}
    if op == "dispatch":
        r = mx.moe_sort(st["experts"], case["e"], align=case["align"])
        return dict(counts=r["counts"], pos=r["pos"], slots=r["slots"],
                    x=mx.moe_gather(st["x"], r["slots"], case["top"]))
    if op == "combine":
        return mx.moe_combine(st["y"], weights=st["weights"], pos=st["pos"])
    r = mx.moe_combine_backward(st["dout"], st["y"], st["weights"], pos=st["pos"], slots=st["slots"])
    return dict(dy=r["dy"], dweights=r["dweights"])


PLAIN = dict(norm=_plain_norm, norm_back=_plain_norm_back, route=_plain_route,
             route_back=_plain_route_back, dispatch=_plain_dispatch, combine=_plain_combine,
             combine_back=_plain_combine_back)


def run(st):
    return _own(st) if own else PLAIN[st["case"]["op"]](st)


# ---- the definition in 64 bits ----------------------------------------------

def _exact_mx(y, fmt, up):
    """Element values and scales of 64-bit values that bf16 holds, along rows."""
    bits, low, top = (3, -6, 448.0) if fmt == "e4m3" else (2, -14, 57344.0)
    R, C = y.shape
    pad = torch.zeros(R, -(-C // 32) * 32, dtype=F64, device=DEV)
    pad[:, :C] = y
    blocks = pad.view(R, -1, 32)
    amax = blocks.abs().amax(2)
    if up:
        power = torch.ceil(torch.log2(amax.clamp_min(1e-300) / top))
    else:
        power = torch.floor(torch.log2(amax.clamp_min(1e-300))) - math.floor(math.log2(top))
    power = power.clamp(-127, 127)
    v = blocks * torch.exp2(-power).unsqueeze(2)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp_min(low) - bits)
    v = (torch.round(v / step) * step).clamp(-top, top)
    return v.reshape(R, -1)[:, :C], torch.exp2(power)


def _exact_scales(s, tiled):
    if not tiled:
        return s
    R, C = s.shape
    RT, CT = (R + 31) // 32, (C + 7) // 8
    word, byte = torch.arange(64, device=DEV).view(1, 1, 64, 1), torch.arange(4, device=DEV)
    row = 32 * torch.arange(RT, device=DEV).view(1, RT, 1, 1) + word % 32
    block = 8 * torch.arange(CT, device=DEV).view(CT, 1, 1, 1) + 2 * byte + word // 32
    inside = (row < R) & (block < C)
    v = s[row.clamp_max(R - 1), block.clamp_max(C - 1)]
    return torch.where(inside, v, torch.full_like(v, 2.0 ** -127)).reshape(-1)


def _exact_norm(st):
    case, o = st["case"], {}
    h = st["x"].double()
    if st["res"] is not None:
        h = h + st["res"].double()
        o["h"] = h
    h = h.to(BF16).double()
    o["rstd"] = ((h * h).sum(1) / case["k"] + 1e-6) ** -0.5
    y = h * o["rstd"].view(-1, 1) * st["w"].double()
    if case["y"]:
        o["y"] = y
    y = y.to(BF16).double()
    for bit, name, v in ((1, "row", y), (2, "col", y.t())):
        if case["axis"] & bit:
            o["q_" + name], s = _exact_mx(v, case["fmt"], case["up"])
            o["s_" + name] = _exact_scales(s, case["tiled"])
    if case["ckpt"]:
        o["q_h"], o["s_h"] = _exact_mx(h, "e4m3", True)
    return o


def _exact_norm_back(st):
    k = st["case"]["k"]
    if st["h"] is None:
        col = torch.arange(k, device=DEV) // 32
        h = st["q_h"].double() * (2.0 ** (st["s_h"].double() - 127))[:, col]
    else:
        h = st["h"].double()
    rstd, dy = st["rstd"].double().view(-1, 1), st["dy"].double()
    gw = dy * st["w"].double()
    # dh = rstd g - rstd^3 h <g, h> / k, from y = h rstd w and d rstd / dh = -rstd^3 h / k
    dh = rstd * gw - rstd ** 3 * h * ((gw * h).sum(1, keepdim=True) / k)
    if st["dres"] is not None:
        dh = dh + st["dres"].double()
    return dict(dh=dh, dweight=(dy * (h * rstd)).sum(0))


def _exact_scores(logits, kind):
    x = logits.double()
    if kind == "sigmoid":
        return torch.sigmoid(x)
    return torch.nan_to_num(torch.softmax(x, 1), nan=0.0)


def _exact_route(st):
    case = st["case"]
    chosen = _plain_route(st)["experts"]     # whole numbers: compared on their own
    p = _exact_scores(st["logits"], case["score"])
    w = torch.where(chosen >= 0, p.gather(1, chosen.clamp_min(0).long()), 0.0)
    if case["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    o = dict(experts=None, weights=w * 2.5)
    if case["scores"]:
        o["scores"] = p
    return o


def _exact_route_back(st):
    """The weights' and scores' derivatives, through the library's autograd in
    64 bits."""
    case = st["case"]
    x = st["logits"].double().requires_grad_(True)
    live = st["experts"] >= 0
    if case["score"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        some = (x > float("-inf")).any(1, keepdim=True)
        p = torch.softmax(torch.where(some, x, torch.zeros_like(x)), 1) * some
    w = torch.where(live, p.gather(1, st["experts"].clamp_min(0).long()), 0.0)
    if case["renorm"]:
        s = w.sum(1, keepdim=True)
        w = w / torch.where(s > 0, s, torch.ones_like(s))
    loss = (2.5 * w * st["dweights"].double()).sum()
    if st["dscores"] is not None:
        loss = loss + (p * st["dscores"].double()).sum()
    g, = torch.autograd.grad(loss, x)
    return torch.nan_to_num(g, nan=0.0)


def _exact_dispatch(st):
    """The rows, expert by expert (whole numbers: compared on their own)."""
    case, at = st["case"], 0
    x = torch.zeros(_capacity(case), case["k"], dtype=F64, device=DEV)
    for e in range(case["e"]):
        token = torch.nonzero((st["experts"] == e).view(-1)).view(-1) // case["top"]
        x[at:at + token.numel()] = st["x"][token].double()
        at += -(-token.numel() // case["align"]) * case["align"]
    return dict(counts=None, pos=None, slots=None, x=x)


def _exact_combine(st):
    case = st["case"]
    out = torch.zeros(case["t"], case["k"], dtype=F64, device=DEV)
    for j in range(case["top"]):
        y = st["y"][:, j] if st["pos"] is None else st["y"][st["pos"][:, j].clamp_min(0).long()]
        w = 1.0 if st["weights"] is None else st["weights"][:, j:j + 1].double()
        live = 1.0 if st["pos"] is None else (st["pos"][:, j:j + 1] >= 0).double()
        out += w * live * y.double()
    return out


def _exact_combine_back(st):
    case, rows = st["case"], _capacity(st["case"])
    dy = torch.zeros(rows, case["k"], dtype=F64, device=DEV)
    dw = torch.zeros(case["t"], case["top"], dtype=F64, device=DEV)
    dout = st["dout"].double()
    for j in range(case["top"]):
        t = torch.nonzero(st["pos"][:, j] >= 0).view(-1)
        r = st["pos"][t, j].long()
        dy[r] = dout[t] * st["weights"][t, j].double().view(-1, 1)
        dw[t, j] = (dout[t] * st["y"][r].double()).sum(1)
    return dict(dy=dy, dweights=dw)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "norm":
        return _exact_norm(st)
    if op == "norm_back":
        return _exact_norm_back(st)
    if op == "route":
        return _exact_route(st)
    if op == "route_back":
        return _exact_route_back(st)
    if op == "dispatch":
        return _exact_dispatch(st)
    if op == "combine":
        return _exact_combine(st)
    return _exact_combine_back(st)
