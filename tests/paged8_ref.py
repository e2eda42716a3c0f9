"""Plain 64-bit forms of the operators over a cache in 8 bits and of the logits processors, and inputs for their tests."""
import math

import numpy as np
import torch

HD = 128
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative
E_MIN, E_MAX = -100, 119


def power(e):
    """2^e in 64 bits, e an int tensor; 128 (the byte 255): NaN."""
    p = ((e.long() + 1023) << 52).view(torch.float64)
    return torch.where(e == 128, math.nan, p)


def decode(codes):
    """e4m3 values in 64 bits of bytes, from the bits."""
    b = codes.view(torch.uint8).long()
    ex, m = (b >> 3) & 15, b & 7
    v = torch.where(ex > 0, (8 + m) * power(ex - 10), m * power(torch.full_like(ex, -9)))
    v = torch.where((b & 0x7f) == 0x7f, math.nan, v)
    return torch.where(b >= 128, -v, v)


def nearest(x, e):
    """x as a code times 2^e: the nearest, ties to even, at most 448."""
    y = x * power(-e)
    step = torch.clamp(torch.frexp(y)[1] - 1, min=-6) - 3
    return ((y * power(-step)).round() * power(step)).clamp(-448, 448) * power(e)


def need(amax):
    """The least e in E_MIN..E_MAX with amax <= 448 * 2^e."""
    e = torch.full(amax.shape, E_MIN, dtype=torch.int32, device=amax.device)
    for t in range(E_MIN, E_MAX):
        e = torch.where(amax > 448 * 2.0 ** t, t + 1, e)
    return e


def make(lens, nq, nkv, page, block, act, seed, extra_rows=0, nhd=False, spare=2, spread=1.0, at_new=False):
    """Pools, table and queries for sequences of (new tokens, context incl. them).  Slots that no sequence owns hold NaN
    codes, blocks without any owned slot a scale of NaN, unused table entries an id far out of range.  spread: scales
    differ by up to 2^spread either way.  at_new: what the new tokens' slots hold is not owned either."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need_p = [-(-c // page) for _, c in lens]
    n_pages = sum(need_p) + spare
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    max_pages = max(need_p + [1]) + 1
    table = torch.full((len(lens), max_pages), 1 << 30, dtype=torch.int32)
    owned = torch.zeros(n_pages, page, dtype=torch.bool)
    at = 0
    for i, (n, c) in enumerate(lens):
        for j in range(need_p[i]):
            table[i, j] = perm[at]
            owned[perm[at], :min(page, max(0, (c - n if at_new else c) - j * page))] = True
            at += 1
    free = (~owned).cuda()
    pools = []
    for _ in range(2):
        # codes of normal values under a scale that the largest of them nearly fills
        x = torch.randn(n_pages, nkv, page, HD, generator=g, device="cuda") * 100
        codes = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes = torch.where(free[:, None, :, None], 0x7f, codes).to(torch.uint8)
        e = (torch.rand(n_pages, nkv, page // block, generator=g, device="cuda") * 2 - 1) * spread - 7
        scale = (e.round() + 127).to(torch.uint8)
        scale = torch.where(owned.cuda().view(n_pages, 1, page // block, block).any(-1), scale, 255).to(torch.uint8)
        if nhd:
            codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
        pools += [codes.view(torch.float8_e4m3fn), scale]
    off = [0]
    for q, _ in lens:
        off.append(off[-1] + q)
    q = torch.randn(off[-1] + extra_rows, nq, HD, generator=g, device="cuda").to(act)
    return {"k": pools[0], "ks": pools[1], "v": pools[2], "vs": pools[3], "table": table.cuda(), "q": q,
            "off": torch.tensor(off, dtype=torch.int32).cuda(),
            "ctx": torch.tensor([c for _, c in lens], dtype=torch.int32).cuda(), "lens": lens, "page": page,
            "block": block, "nq": nq, "nkv": nkv}


def cache_of(s, **kw):
    import speech_lm_decode_gb300 as q3
    return q3.PagedKV8(s["k"], s["v"], s["ks"], s["vs"], s["table"], n_q_heads=s["nq"], **kw)


def values(codes, scale, block):
    """Pages in 64 bits: [pages, nkv, page, 128]."""
    return decode(codes) * power(scale.view(torch.uint8).int() - 127).repeat_interleave(block, -1)[..., None]


def gather(s, i, n):
    """Keys and values of sequence i, positions 0..n-1: [n, nkv, 128] in 64 bits."""
    pages = s["table"][i, :-(-n // s["page"])].long()
    return tuple(values(s[c].view(torch.uint8)[pages], s[c + "s"][pages], s["block"]).transpose(1, 2)
                 .reshape(-1, s["nkv"], HD)[:n] for c in "kv")


def attend64(s, scale=HD ** -0.5):
    """(output, bound of its error per value) for every row, in 64 bits.

    The bound: a score is off by at most scale * sum |q||k| * e_s with e_s = 2^-17 (operand parts) + 2^-17 (128 fp32
    additions); a weight by twice the largest such error, by 2^-17 + 2^-20 (its parts, exp) or, with weights of one
    fp16 part, 2^-11, and by n + 128 additions of 2^-24; each of these multiplies sum p |v|.  The output's own rounding
    comes on top."""
    out, bound = [], []
    act = s["q"].dtype
    for i, (n_new, ctx) in enumerate(s["lens"]):
        rows = s["q"][int(s["off"][i]):int(s["off"][i]) + n_new].double()
        o = torch.zeros(n_new, s["nq"], HD, dtype=torch.float64, device="cuda")
        b = torch.zeros_like(o)
        if ctx > 0 and n_new > 0:
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
                e_p = 2.0 ** -17 + 2.0 ** -20 + (ctx + 128) * 2.0 ** -24 + (2.0 ** -11 if act != torch.float32 else 0)
                b[:, h] = (p @ vh.abs()) * (2 * e_s + e_p)[:, None]
        out.append(o)
        bound.append(b + o.abs() * HALF[act])
    return torch.cat(out), torch.cat(bound)


def turned64(qkv, pos, rope, qn, kn, eps, nq, nkv):
    """(q, its bound), (k, its bound), v of every token in 64 bits: each value is a sum of two products with the normed
    head; the norm's 128 squares, the division and the root cost at most 80 half steps of fp32."""
    x = qkv.double().reshape(-1, nq + 2 * nkv, HD)
    cs = rope.double()[pos.long().clamp(min=0, max=rope.shape[0] - 1)]
    c, d = cs[:, None, :, 0], cs[:, None, :, 1]

    def turn(h, w):
        if w is not None:
            h = h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        a, b = h[..., :64], h[..., 64:]
        y = torch.cat((a * c - b * d, b * c + a * d), -1)
        size = torch.cat((a.abs() * c.abs() + b.abs() * d.abs(), b.abs() * c.abs() + a.abs() * d.abs()), -1)
        return y, size * 80 * 2.0 ** -24
    return turn(x[:, :nq], qn), turn(x[:, nq:nq + nkv], kn), x[:, nq + nkv:]


def check_append(s, before, qkv, rope, qn, kn, eps=1e-6, skip=()):
    """Every block of the pools after an append against the definition, from the pools `before` (clones of k, ks, v, vs);
    skip: (sequence, position) pairs that are not appended.  Returns the bounds of the queries: (q, bound, live)."""
    nq, nkv, page, block = s["nq"], s["nkv"], s["page"], s["block"]
    lens, off = s["lens"], s["off"].tolist()
    pos = torch.cat([torch.arange(c - n, c) for n, c in lens] + [torch.zeros(0, dtype=torch.long)]).cuda()
    (q, qb), (k, kb), v = turned64(qkv[:off[-1]], pos, rope, qn, kn, eps, nq, nkv)
    live = torch.tensor([p >= 0 and (i, p) not in skip for i, (n, c) in enumerate(lens) for p in range(c - n, c)],
                        dtype=torch.bool).cuda()
    n_pages, per = s["k"].shape[0], page // block
    row = torch.full((n_pages, page), -1, dtype=torch.long)       # the token of each slot written
    old = torch.zeros(n_pages, page, dtype=torch.bool)            # older positions of the sequences that are appended to
    at, alive, table = 0, live.tolist(), s["table"].tolist()
    for i, (n, c) in enumerate(lens):
        past = max(0, c - n)
        for j, p in enumerate(range(c - n, c)):
            if alive[at + j]:
                row[table[i][p // page], p % page] = at + j
        if n:
            for p in range(past // block * block, past):
                old[table[i][p // page], p % page] = True
        at += n
    row, old = row.cuda(), old.cuda()
    new = row >= 0
    touched = new.view(n_pages, per, block).any(-1)                                   # [pages, blocks]
    old &= touched.repeat_interleave(block, -1)
    has_old = old.view(n_pages, per, block).any(-1)
    for name, y, b in (("k", k, kb), ("v", v, torch.zeros_like(v))):
        was_c, was_s = before[name], before[name + "s"]
        now_c, now_s = s[name].view(torch.uint8), s[name + "s"]
        e, e0 = now_s.int() - 127, was_s.int() - 127
        assert torch.equal(now_s[~touched[:, None].expand_as(now_s)], was_s[~touched[:, None].expand_as(was_s)])
        keep = ~(new | old)
        assert torch.equal(now_c.transpose(1, 2)[keep], was_c.transpose(1, 2)[keep]), name
        fy, fb = (t[row.clamp(min=0)].transpose(1, 2) for t in (y, b))               # [pages, nkv, page, 128]
        fine = torch.isfinite(fy) & new[:, None, :, None]
        top = lambda t: torch.where(fine, t, 0).amax(-1).view(n_pages, nkv, per, block).amax(-1)  # noqa: E731
        lo, hi = need(top((fy.abs() - fb).clamp(min=0))), need(top(fy.abs() + fb))
        e0 = torch.where(has_old[:, None], e0, -1000)
        t = touched[:, None].expand_as(e)
        assert ((e >= torch.maximum(lo, e0)) & (e <= torch.maximum(hi, e0)))[t].all(), name
        deep = e.repeat_interleave(block, -1)[..., None].expand_as(fy)
        got = decode(now_c) * power(deep)
        n4 = new[:, None, :, None].expand_as(fy)
        below, above = nearest(fy - fb, deep), nearest(fy + fb, deep)
        ok = torch.where(fine, (got >= below) & (got <= above), torch.isnan(got))
        assert ok[n4].all(), (name, torch.nonzero(n4 & ~ok)[:4].tolist())
        o4 = old[:, None, :, None].expand_as(fy)
        base = torch.where(has_old[:, None], was_s.int() - 127, 0).repeat_interleave(block, -1)[..., None].expand_as(fy)
        want = nearest(decode(was_c) * power(base), deep)
        assert torch.equal(got[o4].nan_to_num(7e77), want[o4].nan_to_num(7e77)), name
    return q, qb, live


def process64(x, history=None, n_history=None, n_prompt=None, repetition=None, presence=None, frequency=None,
              bias_off=None, bias_ids=None, bias=None, mask=None, mask_row=None):
    """(result, bound before its own rounding) in 64 bits, numpy: every step rounds once to fp32."""
    n, v = x.shape
    y, size = x.astype(np.float64).copy(), np.abs(x.astype(np.float64))
    for r in range(n):
        if history is not None:
            h = history[r, :max(0, min(int(n_history[r]), history.shape[1]))]
            cut = 0 if n_prompt is None else max(0, min(int(n_prompt[r]), len(h)))
            said = h[cut:]
            h, said = h[(h >= 0) & (h < v)], said[(said >= 0) & (said < v)]
            if repetition is not None:
                for i in set(h.tolist()):
                    f = float(repetition[r]) if y[r, i] < 0 else 1 / float(repetition[r])
                    y[r, i], size[r, i] = y[r, i] * f, size[r, i] * max(1, f)
            for i, c in zip(*np.unique(said, return_counts=True)):
                less = (float(presence[r]) if presence is not None else 0) + c * (float(frequency[r]) if frequency is not None else 0)
                y[r, i] -= less
                size[r, i] += abs(float(presence[r]) if presence is not None else 0) + \
                    c * abs(float(frequency[r]) if frequency is not None else 0)
        if bias_off is not None and 0 <= bias_off[r] <= bias_off[r + 1] <= len(bias):
            inside = [j for j in range(bias_off[r], bias_off[r + 1]) if 0 <= bias_ids[j] < v]
            times = {}
            for j in inside:
                times[bias_ids[j]] = times.get(bias_ids[j], 0) + 1
            for j in inside:
                y[r, bias_ids[j]] += float(bias[j])
                size[r, bias_ids[j]] += times[bias_ids[j]] * abs(float(bias[j]))     # that many sums follow it
        if mask is not None:
            m = r if mask_row is None else int(mask_row[r])
            if m < -1 or m >= len(mask):
                y[r] = -np.inf
            elif m >= 0:
                bits = np.unpackbits(np.ascontiguousarray(mask[m]).view(np.uint8), bitorder="little")[:v]
                y[r][bits == 0] = -np.inf
    return y, size * 6 * 2.0 ** -24
