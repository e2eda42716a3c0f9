"""Plain 64-bit forms of the paged-cache operators and of the draw, and inputs for their tests."""
import math

import numpy as np
import torch

HD = 128
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def make(lens, nq, nkv, page, act, kv, seed, extra_rows=0, nhd=False, spare=2, poison=True):
    """Pools, table and queries for sequences of (new tokens, context incl. them).  Slots that no sequence owns
    hold NaN; unused table entries hold an id far out of range."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    need = [-(-c // page) for _, c in lens]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    max_pages = max(need + [1]) + 1
    table = torch.full((len(lens), max_pages), 1 << 30, dtype=torch.int32)
    shape = (n_pages, page, nkv, HD) if nhd else (n_pages, nkv, page, HD)
    k, v = randn(*shape).to(kv), randn(*shape).to(kv)
    if nhd:
        k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    owned = torch.zeros(n_pages, page, dtype=torch.bool)
    at = 0
    for i, (_, c) in enumerate(lens):
        for j in range(need[i]):
            table[i, j] = perm[at]
            owned[perm[at], :min(page, c - j * page)] = True
            at += 1
    if poison:
        free = (~owned).cuda()[:, None, :, None]
        k.masked_fill_(free, float("nan"))
        v.masked_fill_(free, float("nan"))
    off = [0]
    for q, _ in lens:
        off.append(off[-1] + q)
    return {"k": k, "v": v, "table": table.cuda(), "q": randn(off[-1] + extra_rows, nq, HD).to(act),
            "off": torch.tensor(off, dtype=torch.int32).cuda(),
            "ctx": torch.tensor([c for _, c in lens], dtype=torch.int32).cuda(), "lens": lens, "page": page,
            "nq": nq, "nkv": nkv}


def gather(s, i, n):
    """Keys and values of sequence i, positions 0..n-1: [n, nkv, 128] in 64 bits."""
    pages = s["table"][i, :-(-n // s["page"])].long()
    return tuple(p[pages].transpose(1, 2).reshape(-1, s["nkv"], HD)[:n].double() for p in (s["k"], s["v"]))


def attend64(s, scale=HD ** -0.5):
    """(output, bound of its error per value) for every row, in 64 bits.

    The bound: a score is off by at most scale * sum |q||k| * e_s with e_s = 2^-17 (operand parts) + 2^-17
    (128 fp32 additions); a weight by twice the largest such error, by 2^-17 + 2^-20 (its parts, exp) or, with
    bf16 weights, 2^-8, and by n + 128 additions of 2^-24; each of these multiplies sum p |v|.  The output's own
    rounding comes on top."""
    out, bound = [], []
    act = s["q"].dtype
    for i, (n_new, ctx) in enumerate(s["lens"]):
        rows = s["q"][int(s["off"][i]):int(s["off"][i]) + n_new].double()
        o = torch.zeros(n_new, s["nq"], HD, dtype=torch.float64, device="cuda")
        b = torch.zeros_like(o)
        if ctx > 0:
            k, v = gather(s, i, ctx)
            last = ctx - n_new + torch.arange(n_new, device="cuda")
            future = torch.arange(ctx, device="cuda")[None] > last[:, None]
            some = last >= 0
            for h in range(s["nq"]):
                kh, vh = k[:, h * s["nkv"] // s["nq"]], v[:, h * s["nkv"] // s["nq"]]
                x = (rows[:, h] @ kh.T * scale).masked_fill(future, -math.inf)
                p = torch.softmax(x, -1)
                p[~some] = 0
                o[:, h] = p @ vh
                e_s = scale * (rows[:, h].abs() @ kh.abs().T).masked_fill(future, 0).amax(-1) * 2.0 ** -16
                e_p = 2.0 ** -17 + 2.0 ** -20 + (ctx + 128) * 2.0 ** -24 + (2.0 ** -8 if act != torch.float32 else 0)
                b[:, h] = (p @ vh.abs()) * (2 * e_s + e_p)[:, None]
        out.append(o)
        bound.append(b + o.abs() * HALF[act])
    return torch.cat(out), torch.cat(bound)


def append64(qkv, seq, pos, rope, qn, kn, eps, nq, nkv):
    """(q, k, v) of every token in 64 bits and the bounds of q and k: each value is a sum of two products with
    the normed head; the norm's 128 squares, the division and the root cost at most 80 half steps of fp32."""
    x = qkv.double().reshape(-1, nq + 2 * nkv, HD)
    cs = rope.double()[pos.long().clamp(min=0)]
    c, d = cs[:, None, :, 0], cs[:, None, :, 1]

    def turn(h, w):
        if w is not None:
            h = h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        a, b = h[..., :64], h[..., 64:]
        y = torch.cat((a * c - b * d, b * c + a * d), -1)
        size = torch.cat((a.abs() * c.abs() + b.abs() * d.abs(), b.abs() * c.abs() + a.abs() * d.abs()), -1)
        return y, size * 80 * 2.0 ** -24
    q, qb = turn(x[:, :nq], qn)
    k, kb = turn(x[:, nq:nq + nkv], kn)
    return (q, qb), (k, kb), x[:, nq + nkv:]


F = np.float32


def spec_exp(d):
    """The draw's exp of d <= 0 in single fp32 operations (the definition of its weights)."""
    n = np.rint(d * F(1.44269502162933349609375))
    r = (d - n * F(0.693145751953125)) - n * F(1.428606765330187e-06)
    p = np.full_like(r, F(1 / 40320))
    for c in (1 / 5040, 1 / 720, 1 / 120, 1 / 24, 1 / 6, 0.5, 1, 1):
        p = F(c) + r * p
    return np.where(d < F(-86), F(0), np.ldexp(p, n.astype(np.int32))).astype(F)


def draw_row(x, u, t, k, top_p, min_p):
    """(id, log probability, its bound) of one row; x float32."""
    if not t >= 0:
        return -1, math.nan, 0
    with np.errstate(all="ignore"):
        l = x / F(t) if t > 0 else x
    if np.isnan(l).any() or (l == np.inf).any() or (l == -np.inf).all():
        return -1, math.nan, 0
    first = int(np.argmax(l))
    if t == 0:
        return first, 0.0, 0
    m = l[first]
    e = np.zeros_like(l)
    fine = np.isfinite(l)
    e[fine] = spec_exp(l[fine] - m)
    w = np.floor(np.ldexp(e.astype(np.float64), 40)).astype(np.int64)
    in_k = l >= np.sort(l)[-k] if 0 < k < len(l) else np.ones(len(l), bool)
    order = np.lexsort((np.arange(len(l)), -l))
    order = order[in_k[order]]
    keep = np.zeros(len(l), bool)
    if top_p >= 1:
        keep[order] = True
    else:
        total = float(int(w[order].sum()))
        before = 0
        for j in order:
            if not float(before) < float(F(top_p)) * total:
                break
            keep[j] = True
            before += int(w[j])
    keep &= e >= F(min_p)
    keep[first] = True
    upto = np.cumsum(np.where(keep, w, 0))
    z = int(upto[-1])
    target = min(int(float(u) * float(z)), z - 1) if u > 0 else 0
    i = int(np.searchsorted(upto, target, side="right"))
    a, b = float(l[i]) - float(m), math.log(z * 2.0 ** -40)
    return i, a - b, 2.0 ** -23 * (abs(a) + abs(b)) + 2.0 ** -40
