"""Cases of the paged-cache serving operators and of the draw from given random numbers.

Three operators, as one serving step uses them: appending keys and values to a paged cache with the norms of each
head and the rotation on the way ("append"), attention of the new tokens over that cache ("attend"), and the draw
from logits with temperature, top-k, top-p and min-p ("draw").  `run` computes them in plain torch operations, or,
with `own`, through speech_lm_decode_gb300.
"""
import math
import random

import torch

own = False

HD = 128        # head dimension
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence: the batch-1 decode step, where latency is all
        {"name": "append-1", "op": "append", "seqs": 1, "q_lo": 1, "q_hi": 1, "past_lo": 227, "past_hi": 227, "nq": 16,
         "nkv": 8, "page": 16, "act": "f32", "kv": "bf16", "norm": True, "shape": 1},
        # a decode step of a large batch: one token for each of 256 sequences
        {"name": "append-256", "op": "append", "seqs": 256, "q_lo": 1, "q_hi": 1, "past_lo": 256, "past_hi": 1279,
         "nq": 16, "nkv": 8, "page": 16, "act": "f32", "kv": "bf16", "norm": True, "shape": 2},
        # prompts of 32 sequences in one pass, bf16 activations
        {"name": "append-prompts", "op": "append", "seqs": 32, "q_lo": 64, "q_hi": 512, "past_lo": 0, "past_hi": 0,
         "nq": 16, "nkv": 8, "page": 32, "act": "bf16", "kv": "bf16", "norm": True, "shape": 3},
        # the batch-1 decode step over a short context
        {"name": "attend-1", "op": "attend", "seqs": 1, "q_lo": 1, "q_hi": 1, "past_lo": 227, "past_hi": 227, "nq": 16,
         "nkv": 8, "page": 16, "act": "bf16", "kv": "bf16", "shape": 4},
        # 32 sequences of unlike lengths, fp32 activations, as the frame loop holds them
        {"name": "attend-32-ragged", "op": "attend", "seqs": 32, "q_lo": 1, "q_hi": 1, "past_lo": 64, "past_hi": 767,
         "nq": 16, "nkv": 8, "page": 16, "act": "f32", "kv": "bf16", "shape": 5},
        # 256 sequences near the end of a long generation
        {"name": "attend-256", "op": "attend", "seqs": 256, "q_lo": 1, "q_hi": 1, "past_lo": 1024, "past_hi": 1279,
         "nq": 16, "nkv": 8, "page": 64, "act": "bf16", "kv": "bf16", "shape": 6},
        # few sequences with long caches and eight query heads to a key head
        {"name": "attend-long", "op": "attend", "seqs": 3, "q_lo": 1, "q_hi": 1, "past_lo": 30001, "past_hi": 65537,
         "nq": 32, "nkv": 4, "page": 64, "act": "bf16", "kv": "bf16", "shape": 7},
        # a chunk of a long prompt over what the cache holds already
        {"name": "attend-chunk", "op": "attend", "seqs": 1, "q_lo": 4096, "q_hi": 4096, "past_lo": 12288,
         "past_hi": 12288, "nq": 16, "nkv": 8, "page": 64, "act": "bf16", "kv": "bf16", "shape": 8},
        # prompts of a batch in one pass, fp32 activations; a few rows are a single token
        {"name": "attend-prompts", "op": "attend", "seqs": 24, "q_lo": 1, "q_hi": 512, "past_lo": 0, "past_hi": 255,
         "nq": 16, "nkv": 8, "page": 16, "act": "f32", "kv": "bf16", "shape": 9},
        # one draw over a codebook
        {"name": "draw-1", "op": "draw", "rows": 1, "vocab": 2048, "logits": "f32", "top_k": 50, "top_p": 1.0,
         "min_p": 0.0},
        # a batch over a text vocabulary, every filter on
        {"name": "draw-32-text", "op": "draw", "rows": 32, "vocab": 151936, "logits": "f32", "top_k": 50,
         "top_p": 0.95, "min_p": 0.02},
        # a large batch over a text vocabulary, top-p over all of it, bf16 logits
        {"name": "draw-256-text", "op": "draw", "rows": 256, "vocab": 151936, "logits": "bf16", "top_k": 0,
         "top_p": 0.95, "min_p": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "draw"))
    if op == "draw":
        vocab = _log(rng, 33, 200000)
        return {"op": op, "rows": max(1, min(_log(rng, 1, 512), 256 * 151936 // vocab)), "vocab": vocab,
                "logits": rng.choice(("f32", "bf16")), "top_k": rng.choice((0, 1, 20, 50, 400)),
                "top_p": rng.choice((1.0, 0.95, 0.8, 0.5)), "min_p": rng.choice((0.0, 0.0, 0.02, 0.1))}
    act, kv = rng.choice((("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")))
    nq, nkv = rng.choice(((16, 8), (16, 8), (16, 4), (32, 8), (28, 4), (8, 8), (16, 1)))
    seqs = _log(rng, 1, 256)
    top = rng.choice((1, 1, 4, _log(rng, 2, 2048)))          # new tokens of a sequence, at most
    top = max(1, min(top, 8192 // seqs))
    past = _log(rng, 1, max(2, min(32768, 262144 // seqs)))
    if op == "attend":
        # the plain form's scores and the kernels' products stay below the largest listed case
        past = max(1, min(past, 2 ** 28 // max(1, seqs * nq * top) - top, 2 ** 25 // max(1, seqs * nkv)))
    c = {"op": op, "seqs": seqs, "q_lo": rng.choice((1, max(1, top // 2), top)), "q_hi": top,
         "past_lo": rng.choice((0, past // 2, past)), "past_hi": past, "nq": nq, "nkv": nkv,
         "page": rng.choice((16, 32, 64, 128)), "act": act, "kv": kv, "shape": rng.randrange(1 << 20)}
    if op == "append":
        c["norm"] = rng.choice((True, True, False))
    return c


def _lengths(case):
    """(new tokens, tokens cached before them) of each sequence; they go by the case alone."""
    r = random.Random(case["shape"])
    return [(r.randint(case["q_lo"], case["q_hi"]), r.randint(case["past_lo"], case["past_hi"]))
            for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "draw":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * SIZE[case["logits"]] + case["rows"] * 28, "flops": 10 * n}
    lens = _lengths(case)
    m = sum(q for q, _ in lens)
    nq, nkv, ea, ek = case["nq"], case["nkv"], SIZE[case["act"]], SIZE[case["kv"]]
    if case["op"] == "append":
        return {"bytes": m * ((2 * nq + 2 * nkv) * HD * ea + 2 * nkv * HD * ek + HD // 2 * 8 + 8),
                "flops": m * (nq + nkv) * HD * 7}
    keys = sum(q + p for q, p in lens)
    pairs = sum(q * p + q * (q + 1) // 2 for q, p in lens)
    return {"bytes": keys * nkv * HD * 2 * ek + 2 * m * nq * HD * ea, "flops": 4 * HD * nq * pairs}


# ---------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "draw":
        n, v = case["rows"], case["vocab"]
        logits = _randn(g, n, v, scale=2.5)
        # ids that a serving program never draws
        logits[:, torch.randint(0, v, (v // 64,), generator=g, device="cuda")] = float("-inf")
        logits[:, v // 2] = 1.0
        s["logits"] = logits.to(DT[case["logits"]])
        s["u"] = torch.rand(n, generator=g, device="cuda")
        s["temperature"] = 0.6 + 0.6 * torch.rand(n, generator=g, device="cuda")
        s["top_k"] = torch.full((n,), case["top_k"], dtype=torch.int32, device="cuda")
        s["top_p"] = torch.full((n,), case["top_p"], dtype=torch.float32, device="cuda")
        s["min_p"] = torch.full((n,), case["min_p"], dtype=torch.float32, device="cuda")
        if own:
            import speech_lm_decode_gb300 as q3
            s["sample"] = q3.sample_given
        return s
    lens = _lengths(case)
    page, nq, nkv = case["page"], case["nq"], case["nkv"]
    act, kv = DT[case["act"]], DT[case["kv"]]
    need = [-(-(q + p) // page) for q, p in lens]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32)
    # pages of a sequence lie anywhere in the pool
    at, order = 0, perm.cpu()
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    s["table"] = table.cuda()
    s["k_pages"] = _randn(g, n_pages, nkv, page, HD, dtype=kv)
    s["v_pages"] = _randn(g, n_pages, nkv, page, HD, dtype=kv)
    m = sum(q for q, _ in lens)
    s["nq"], s["nkv"], s["page"] = nq, nkv, page
    if case["op"] == "append":
        seq = torch.tensor([i for i, (q, _) in enumerate(lens) for _ in range(q)], dtype=torch.int32)
        pos = torch.tensor([p + j for q, p in lens for j in range(q)], dtype=torch.int32)
        s["seq"], s["pos"] = seq.cuda(), pos.cuda()
        s["qkv"] = _randn(g, m, (nq + 2 * nkv) * HD, dtype=act, scale=1.3)
        rows = max(q + p for q, p in lens)
        # the rotation's table: cosine and sine of position * theta^(-2j/128), angles in 64 bits
        ang = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * \
            (1e6 ** (-torch.arange(HD // 2, device="cuda", dtype=torch.float64) * 2 / HD))[None]
        s["rope"] = torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()
        s["q_norm"] = 1 + _randn(g, HD, scale=0.1) if case["norm"] else None
        s["k_norm"] = 1 + _randn(g, HD, scale=0.1) if case["norm"] else None
    else:
        s["q"] = _randn(g, m, nq, HD, dtype=act, scale=1.5)
        off = [0]
        for q, _ in lens:
            off.append(off[-1] + q)
        s["q_off"] = torch.tensor(off, dtype=torch.int32).cuda()
        s["ctx"] = torch.tensor([q + p for q, p in lens], dtype=torch.int32).cuda()
        s["max_q"] = max(q for q, _ in lens)
        s["max_ctx"] = max(q + p for q, p in lens)
    if own:
        import speech_lm_decode_gb300 as q3
        s["cache"] = q3.PagedKV(s["k_pages"], s["v_pages"], s["table"], n_q_heads=nq)
    return s


# ---------------------------------------------------------------- the plain forms
def run(s):
    if s["op"] == "append":
        if own:
            q = s["cache"].append(s["qkv"], s["seq"], s["pos"], s["rope"], s["q_norm"], s["k_norm"], eps=1e-6)
        else:
            q = _append(s)
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["op"] == "attend":
        if own:
            return s["cache"].attend(s["q"], s["q_off"], s["ctx"], s["max_q"])
        return _attend(s)
    if own:
        ids, logprob = s["sample"](s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    else:
        ids, logprob = _draw(s)
    return {"ids": ids, "logprob": logprob}


def _rms_rope(x, w, cs):
    """Norm of each head's 128 values (w None: none), then the rotation of the pairs (j, j + 64)."""
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    a, b = x[..., :HD // 2], x[..., HD // 2:]
    c, d = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat((a * c - b * d, b * c + a * d), -1)


def _append(s):
    nq, nkv, page = s["nq"], s["nkv"], s["page"]
    m = s["qkv"].shape[0]
    x = s["qkv"].float().view(m, nq + 2 * nkv, HD)
    pos, seq = s["pos"].long(), s["seq"].long()
    cs = s["rope"][pos]
    q = _rms_rope(x[:, :nq], s["q_norm"], cs)
    k = _rms_rope(x[:, nq:nq + nkv], s["k_norm"], cs)
    at, slot = s["table"][seq, pos // page].long(), pos % page
    s["k_pages"][at, :, slot] = k.to(s["k_pages"].dtype)
    s["v_pages"][at, :, slot] = x[:, nq + nkv:].to(s["v_pages"].dtype)
    return q.to(s["qkv"].dtype)


def _attend(s):
    nq, nkv, page = s["nq"], s["nkv"], s["page"]
    b, t, n = s["ctx"].shape[0], s["max_q"], s["max_ctx"]
    off, ctx = s["q_off"].long(), s["ctx"].long()
    count = off[1:] - off[:-1]
    j = torch.arange(n, device="cuda")
    # keys and values of each sequence side by side, [b, n, nkv, 128]
    at = s["table"][:, j // page].long()
    k = s["k_pages"][at, :, j % page].float()
    v = s["v_pages"][at, :, j % page].float()
    i = torch.arange(t, device="cuda")
    there = i[None] < count[:, None]
    rows = (off[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(b, t, nkv, nq // nkv, HD)
    score = torch.einsum("bthgd,bnhd->bhgtn", q, k) * (1 / math.sqrt(HD))
    last = ctx[:, None] - count[:, None] + i[None]            # the position of each new token
    seen = j[None, None] <= last[:, :, None]
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    del score
    o = torch.einsum("bhgtn,bnhd->bthgd", p, v) / p.sum(-1).permute(0, 3, 1, 2)[..., None]
    return o.reshape(b, t, nq, HD)[there].to(s["q"].dtype)


def _exp(x):
    """exp of x <= 0 as the operator defines it, in single IEEE operations: reduction by ln 2 in two parts, a
    Taylor polynomial of degree 8, zero below -86."""
    n = torch.round(x.clamp(min=-87.0) * 1.44269502162933349609375)
    r = x.clamp(min=-87.0) - n * 0.693145751953125
    r = r - n * 1.428606765330187e-06
    p = torch.full_like(r, 1.0 / 40320.0)
    for c in (1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0):
        p = torch.tensor(c, dtype=torch.float32, device=x.device) + r * p
    scale = ((n.int() + 127) << 23).view(torch.float32)
    return torch.where(x < -86.0, torch.zeros_like(p), p * scale)


def _draw(s):
    temp, u = s["temperature"], s["u"]
    x = s["logits"].float()
    greedy = temp == 0
    x = x / torch.where(greedy, torch.ones_like(temp), temp)[:, None]
    v = x.shape[1]
    top, order = torch.sort(x, dim=1, descending=True, stable=True)     # ties: the lowest id first
    bad = torch.isnan(x).any(1) | ~torch.isfinite(top[:, 0])
    k = s["top_k"].long()
    k = torch.where((k <= 0) | (k > v), v, k)
    kth = top.gather(1, k[:, None] - 1)
    e = _exp(top - top[:, :1])
    weight = torch.where(top >= kth, torch.floor(e.double() * 2.0 ** 40), 0.0).long()
    upto = weight.cumsum(1)
    total = upto[:, -1:]
    limit = s["top_p"].double()[:, None] * total.double()
    keep = ((upto - weight).double() < limit) | (s["top_p"] >= 1)[:, None]
    keep &= e >= s["min_p"][:, None]
    keep[:, 0] = True
    kept = torch.zeros_like(weight).scatter_(1, order, torch.where(keep, weight, 0))
    upto = kept.cumsum(1)
    total = upto[:, -1:]
    target = torch.minimum(torch.floor(u.double()[:, None] * total.double()).long(), total - 1)
    ids = (upto <= target).sum(1)
    ids = torch.where(greedy, order[:, 0], ids)
    z = torch.log(total[:, 0].double() * 2.0 ** -40)
    logprob = (x.gather(1, ids.clamp(max=v - 1)[:, None])[:, 0] - top[:, 0]).double() - z
    logprob = torch.where(greedy, 0.0, logprob)
    return (torch.where(bad, -1, ids).to(torch.int32),
            torch.where(bad, float("nan"), logprob).float())


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_draw(s)


def _exact_append(case, s):
    nq, nkv, page = case["nq"], case["nkv"], case["page"]
    x = s["qkv"].double().reshape(-1, nq + 2 * nkv, HD)
    cos, sin = s["rope"].double()[s["pos"].long()].unbind(-1)

    def turned(h, w):
        if w is not None:
            h = h * (h.square().sum(-1, keepdim=True) / HD + 1e-6).rsqrt() * w.double()
        z = torch.complex(h[..., :64].contiguous(), h[..., 64:].contiguous()) * torch.complex(cos, sin)[:, None]
        return torch.cat((z.real, z.imag), -1)
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    k = turned(x[:, nq:nq + nkv], s["k_norm"])
    first = 0
    for i, (q, p) in enumerate(_lengths(case)):
        for j in range(p // page, -(-(q + p) // page)):
            a, b = max(p, j * page), min(q + p, (j + 1) * page)
            src = slice(first + a - p, first + b - p)
            at = int(s["table"][i, j])
            k_pages[at, :, a - j * page:b - j * page] = k[src].transpose(0, 1)
            v_pages[at, :, a - j * page:b - j * page] = x[src, nq + nkv:].transpose(0, 1)
        first += q
    return {"q": turned(x[:, :nq], s["q_norm"]).reshape(-1, nq, HD), "k_pages": k_pages, "v_pages": v_pages}


def _exact_attend(case, s):
    nq, nkv = case["nq"], case["nkv"]
    out, first = [], 0
    for i, (q, p) in enumerate(_lengths(case)):
        n = q + p
        pages = s["table"][i, :-(-n // case["page"])].long()
        k = s["k_pages"][pages].transpose(1, 2).reshape(-1, nkv, HD)[:n].double()
        v = s["v_pages"][pages].transpose(1, 2).reshape(-1, nkv, HD)[:n].double()
        x = s["q"][first:first + q].double()
        future = torch.ones(q, n, dtype=torch.bool, device="cuda").triu(p + 1)
        o = torch.empty(q, nq, HD, dtype=torch.float64, device="cuda")
        for h in range(nq):
            kv = h * nkv // nq
            a = (x[:, h] @ k[:, kv].T / HD ** 0.5).masked_fill(future, -math.inf)
            o[:, h] = torch.softmax(a, -1) @ v[:, kv]
        out.append(o)
        first += q
    return torch.cat(out)


def _exact_draw(s):
    import numpy as np
    f = np.float32
    ids, logprob = [], []
    for x, t, u, k, p, mp in zip(s["logits"].float().cpu().numpy(), *(s[n].cpu().numpy() for n in (
            "temperature", "u", "top_k", "top_p", "min_p"))):
        # the weights are whole numbers by definition: 2^40 times an exp in single IEEE operations, rounded down
        l = x / t
        m = l.max()
        kth = np.partition(l, -k)[-k] if 0 < k < len(l) else -np.inf
        idx = np.flatnonzero((l >= kth) & (l - m >= f(-86)))
        d = l[idx] - m
        n = np.rint(d * f(1.44269502162933349609375))
        r = (d - n * f(0.693145751953125)) - n * f(1.428606765330187e-06)
        e = np.full_like(r, f(1 / 40320))
        for c in (1 / 5040, 1 / 720, 1 / 120, 1 / 24, 1 / 6, 0.5, 1, 1):
            e = f(c) + r * e
        e = np.ldexp(e, n.astype(np.int32))
        w = np.floor(np.ldexp(e.astype(np.float64), 40)).astype(np.int64)
        if p < 1:
            by = np.lexsort((idx, -l[idx]))
            before = np.cumsum(w[by]) - w[by]
            by = by[(before < float(p) * float(w.sum())) | (np.arange(len(by)) == 0)]
            by.sort()
            idx, e, w = idx[by], e[by], w[by]
        idx, w = idx[e >= mp], w[e >= mp]
        upto = np.cumsum(w)
        i = idx[np.searchsorted(upto, min(int(float(u) * float(upto[-1])), int(upto[-1]) - 1), side="right")]
        ids.append(int(i))
        logprob.append(float(l[i]) - float(m) - math.log(float(upto[-1]) * 2.0 ** -40))
    return {"ids": torch.tensor(ids, dtype=torch.int32), "logprob": torch.tensor(logprob, dtype=torch.float64)}
