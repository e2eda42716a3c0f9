"""Cases of the 8-bit paged cache and of the logits processors.

The operators of one serving step over a cache held in 8 bits: appending keys and values to it, quantised in blocks of
tokens with a power-of-two scale for each block and head, and reading back the pages written ("append8"); attention of
the new tokens over it ("attend8"); penalties, biases and grammar masks on the logits in front of the draw
("process").  `run` computes them in plain torch operations, or, with `own`, through speech_lm_decode_gb300.
"""
import math
import random

import torch

own = False

HD = 128        # head dimension
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
E_MIN, E_MAX = -100, 119      # exponents that a block's scale may have


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence: the batch-1 decode step, where latency is all
        {"name": "append8-1", "op": "append8", "seqs": 1, "q_lo": 1, "q_hi": 1, "past_lo": 227, "past_hi": 227,
         "nq": 16, "nkv": 8, "page": 16, "block": 16, "act": "f32", "norm": True, "shape": 1},
        # a decode step of a large batch: one token for each of 256 sequences, blocks that grow
        {"name": "append8-256", "op": "append8", "seqs": 256, "q_lo": 1, "q_hi": 1, "past_lo": 0, "past_hi": 1023,
         "nq": 16, "nkv": 8, "page": 16, "block": 16, "act": "bf16", "norm": True, "shape": 2},
        # prompts of 32 sequences in one pass, in blocks of half a page
        {"name": "append8-prompts", "op": "append8", "seqs": 32, "q_lo": 64, "q_hi": 512, "past_lo": 0, "past_hi": 0,
         "nq": 16, "nkv": 8, "page": 32, "block": 16, "act": "bf16", "norm": True, "shape": 3},
        # the batch-1 decode step over a short context
        {"name": "attend8-1", "op": "attend8", "seqs": 1, "q_lo": 1, "q_hi": 1, "past_lo": 227, "past_hi": 227,
         "nq": 16, "nkv": 8, "page": 16, "block": 16, "act": "bf16", "shape": 4},
        # 32 sequences of unlike lengths, fp32 activations, as the frame loop holds them
        {"name": "attend8-32-ragged", "op": "attend8", "seqs": 32, "q_lo": 1, "q_hi": 1, "past_lo": 64, "past_hi": 767,
         "nq": 16, "nkv": 8, "page": 16, "block": 16, "act": "f32", "shape": 5},
        # 256 sequences near the end of a long generation
        {"name": "attend8-256", "op": "attend8", "seqs": 256, "q_lo": 1, "q_hi": 1, "past_lo": 1024, "past_hi": 1279,
         "nq": 16, "nkv": 8, "page": 64, "block": 64, "act": "bf16", "shape": 6},
        # few sequences with long caches and eight query heads to a key head
        {"name": "attend8-long", "op": "attend8", "seqs": 3, "q_lo": 1, "q_hi": 1, "past_lo": 30001, "past_hi": 65537,
         "nq": 32, "nkv": 4, "page": 64, "block": 32, "act": "bf16", "shape": 7},
        # a chunk of a long prompt over what the cache holds already
        {"name": "attend8-chunk", "op": "attend8", "seqs": 1, "q_lo": 4096, "q_hi": 4096, "past_lo": 12288,
         "past_hi": 12288, "nq": 16, "nkv": 8, "page": 64, "block": 16, "act": "bf16", "shape": 8},
        # prompts of a batch in one pass, fp32 activations; a few rows are a single token
        {"name": "attend8-prompts", "op": "attend8", "seqs": 24, "q_lo": 1, "q_hi": 512, "past_lo": 0, "past_hi": 255,
         "nq": 16, "nkv": 8, "page": 16, "block": 16, "act": "f32", "shape": 9},
        # the penalty on one codebook's logits
        {"name": "process-1", "op": "process", "rows": 1, "vocab": 2048, "logits": "f32", "history": 200, "prompt": 0,
         "biases": 0, "masks": 0, "shape": 10},
        # a batch over a text vocabulary with everything on: histories with their prompts, biases, a few grammars
        {"name": "process-32-text", "op": "process", "rows": 32, "vocab": 151936, "logits": "f32", "history": 2048,
         "prompt": 1024, "biases": 64, "masks": 5, "shape": 11},
        # a large batch over a text vocabulary, bf16 logits, a mask for every row
        {"name": "process-256-text", "op": "process", "rows": 256, "vocab": 151936, "logits": "bf16", "history": 1024,
         "prompt": 512, "biases": 16, "masks": 256, "shape": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append8", "attend8", "attend8", "process"))
    shape = rng.randrange(1 << 20)
    if op == "process":
        vocab = _log(rng, 33, 200000)
        rows = max(1, min(_log(rng, 1, 512), 256 * 151936 // vocab))
        history = rng.choice((0, _log(rng, 1, 16384), _log(rng, 1, 2048)))
        return {"op": op, "rows": rows, "vocab": vocab, "logits": rng.choice(("f32", "bf16")), "history": history,
                "prompt": rng.choice((0, history // 2, history)), "biases": rng.choice((0, min(vocab, _log(rng, 1, 512)))),
                "masks": rng.choice((0, 1, rows)), "shape": shape}
    nq, nkv = rng.choice(((16, 8), (16, 8), (16, 4), (32, 8), (28, 4), (8, 8), (16, 1)))
    seqs = _log(rng, 1, 256)
    top = rng.choice((1, 1, 4, _log(rng, 2, 2048)))          # new tokens of a sequence, at most
    top = max(1, min(top, 8192 // seqs))
    past = _log(rng, 1, max(2, min(32768, 262144 // seqs)))
    if op == "attend8":
        # the plain form's scores and the kernels' products stay below the largest listed case
        past = max(1, min(past, 2 ** 28 // max(1, seqs * nq * top) - top, 2 ** 25 // max(1, seqs * nkv)))
    page = rng.choice((16, 32, 64, 128))
    c = {"op": op, "seqs": seqs, "q_lo": rng.choice((0, 1, max(1, top // 2), top)), "q_hi": top,
         "past_lo": rng.choice((0, past // 2, past)), "past_hi": past, "nq": nq, "nkv": nkv, "page": page,
         "block": rng.choice([b for b in (16, 32, 64, 128) if b <= page]), "act": rng.choice(("bf16", "f32")),
         "shape": shape}
    if op == "append8":
        c["norm"] = rng.choice((True, True, False))
    return c


def _lengths(case):
    """(new tokens, tokens cached before them) of each sequence; they go by the case alone."""
    r = random.Random(case["shape"])
    lens = [(r.randint(case["q_lo"], case["q_hi"]), r.randint(case["past_lo"], case["past_hi"]))
            for _ in range(case["seqs"])]
    if not any(q for q, _ in lens):
        lens[0] = (case["q_hi"], lens[0][1])
    return lens


def _histories(case):
    """(tokens, prompt tokens among them, biases) of each row; they go by the case alone."""
    r = random.Random(case["shape"])
    got = []
    for _ in range(case["rows"]):
        n = r.randint(case["history"] // 2, case["history"])
        got.append((n, min(n, r.randint(case["prompt"] // 2, case["prompt"])), r.randint(0, case["biases"])))
    if case["rows"] == 1:
        got[0] = (case["history"], case["prompt"], case["biases"])
    return got


def _written(case):
    """Pages of each sequence that its new tokens lie in: (sequence, entry of its table)."""
    return [(i, j) for i, (q, p) in enumerate(_lengths(case)) if q
            for j in range(p // case["page"], -(-(q + p) // case["page"]))]


def work(case):
    if case["op"] == "process":
        n = case["rows"] * case["vocab"]
        lens = _histories(case)
        mask = case["masks"] * (-(-case["vocab"] // 32)) * 4
        return {"bytes": 2 * n * SIZE[case["logits"]] + mask + sum(4 * h + 8 * b for h, _, b in lens) + case["rows"] * 28,
                "flops": 3 * n}
    lens = _lengths(case)
    m = sum(q for q, _ in lens)
    nq, nkv, ea = case["nq"], case["nkv"], SIZE[case["act"]]
    if case["op"] == "append8":
        back = len(_written(case)) * case["page"] * nkv * HD * 2 * 3       # codes in, bf16 values out
        return {"bytes": m * ((2 * nq + 2 * nkv) * HD * ea + 2 * nkv * HD + HD // 2 * 8) + back,
                "flops": m * (nq + 2 * nkv) * HD * 7}
    keys = sum(q + p for q, p in lens if q)
    pairs = sum(q * p + q * (q + 1) // 2 for q, p in lens)
    return {"bytes": keys * nkv * (HD * 2 + 2 / case["block"]) + 2 * m * nq * HD * ea, "flops": 4 * HD * nq * pairs}


# ---------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _pool(g, n_pages, nkv, page, block):
    """Pages of codes and their scales (as bytes, the exponent + 127): normal values, heads of unlike size."""
    x = _randn(g, n_pages, nkv, page // block, block * HD)
    x *= torch.exp2(2 * torch.rand(nkv, generator=g, device="cuda") - 1)[:, None, None]
    e = torch.ceil(torch.log2(x.abs().amax(-1) / 448))
    x *= _two(-e)[..., None]
    codes = x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(n_pages, nkv, page, HD)
    return codes, (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "process":
        return _prepare_process(case, g, s)
    lens = _lengths(case)
    page, block, nq, nkv, act = case["page"], case["block"], case["nq"], case["nkv"], DT[case["act"]]
    need = [-(-(q + p) // page) for q, p in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32)
    # pages of a sequence lie anywhere in the pool
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    s["table"] = table.cuda()
    s["k_pages"], k_scale = _pool(g, n_pages, nkv, page, block)
    s["v_pages"], v_scale = _pool(g, n_pages, nkv, page, block)
    s["k_scale"], s["v_scale"] = k_scale.view(torch.float8_e8m0fnu), v_scale.view(torch.float8_e8m0fnu)
    s["nq"], s["nkv"], s["page"], s["block"] = nq, nkv, page, block
    m = sum(q for q, _ in lens)
    off = [0]
    for q, _ in lens:
        off.append(off[-1] + q)
    s["q_off"] = torch.tensor(off, dtype=torch.int32).cuda()
    s["ctx"] = torch.tensor([q + p for q, p in lens], dtype=torch.int32).cuda()
    s["max_q"] = max(q for q, _ in lens)
    s["max_ctx"] = max(q + p for q, p in lens)
    if case["op"] == "append8":
        s["qkv"] = _randn(g, m, (nq + 2 * nkv) * HD, dtype=act, scale=1.3)
        # the rotation's table: cosine and sine of position * theta^(-2j/128), angles in 64 bits
        ang = torch.arange(s["max_ctx"], device="cuda", dtype=torch.float64)[:, None] * \
            (1e6 ** (-torch.arange(HD // 2, device="cuda", dtype=torch.float64) * 2 / HD))[None]
        s["rope"] = torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()
        s["q_norm"] = 1 + _randn(g, HD, scale=0.1) if case["norm"] else None
        s["k_norm"] = 1 + _randn(g, HD, scale=0.1) if case["norm"] else None
        s["pages"] = torch.tensor([int(table[i, j]) for i, j in _written(case)], dtype=torch.int32).cuda()
    else:
        s["q"] = _randn(g, m, nq, HD, dtype=act, scale=1.5)
    if own:
        import speech_lm_decode_gb300 as q3
        s["cache"] = q3.PagedKV8(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], n_q_heads=nq)
    return s


def _prepare_process(case, g, s):
    n, v = case["rows"], case["vocab"]
    lens = _histories(case)
    s["logits"] = _randn(g, n, v, dtype=DT[case["logits"]], scale=2.5)
    names = ("history", "n_history", "n_prompt", "repetition", "presence", "frequency", "bias_off", "bias_ids", "bias",
             "mask", "mask_row")
    s.update({name: None for name in names})
    if case["history"]:
        # tokens repeat: low ids far more often than high ones
        u = torch.rand(n, case["history"], generator=g, device="cuda")
        s["history"] = (u ** 3 * v).long().clamp(max=v - 1).to(torch.int32)
        s["n_history"] = torch.tensor([h for h, _, _ in lens], dtype=torch.int32).cuda()
        s["n_prompt"] = torch.tensor([p for _, p, _ in lens], dtype=torch.int32).cuda()
        s["repetition"] = 1 + 0.3 * torch.rand(n, generator=g, device="cuda")
        s["presence"] = torch.rand(n, generator=g, device="cuda")
        s["frequency"] = 0.5 * torch.rand(n, generator=g, device="cuda")
    if case["biases"]:
        off, ids = [0], []
        r = random.Random(case["shape"])
        for _, _, b in lens:
            step, start = max(1, v // max(1, b)), r.randrange(v)
            ids += [(start + j * step + r.randrange(step)) % v for j in range(b)]
            off.append(off[-1] + b)
        s["bias_off"] = torch.tensor(off, dtype=torch.int32).cuda()
        s["bias_ids"] = torch.tensor(ids, dtype=torch.int32).cuda()
        s["bias"] = _randn(g, len(ids), scale=3.0)
    if case["masks"]:
        m, words = case["masks"], -(-v // 32)
        w = torch.randint(-2 ** 31, 2 ** 31, (3, m, words), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        # grammars that leave most ids and grammars that leave few
        few = torch.rand(m, generator=g, device="cuda") < 0.5
        s["mask"] = torch.where(few[:, None], w[0] & w[1] & w[2], w[0] | w[1] | w[2])
        if m != n:
            s["mask_row"] = torch.randint(-1, m, (n,), generator=g, device="cuda", dtype=torch.int32)
    if own:
        import speech_lm_decode_gb300 as q3
        s["process"] = q3.process_logits
    return s


# ---------------------------------------------------------------- the plain forms
def run(s):
    if s["op"] == "append8":
        if own:
            c = s["cache"]
            q = c.append(s["qkv"], s["q_off"], s["ctx"], s["max_q"], s["rope"], s["q_norm"], s["k_norm"], eps=1e-6)
            k, v = c.read(s["pages"])
        else:
            q = _append(s)
            k, v = (_read(s[n + "_pages"], s[n + "_scale"], s["pages"], s["block"]) for n in "kv")
        # the values that the pages written hold now, and the tokens' queries
        return {"q": q, "k": k, "v": v}
    if s["op"] == "attend8":
        if own:
            return s["cache"].attend(s["q"], s["q_off"], s["ctx"], s["max_q"])
        return _attend(s)
    if own:
        return s["process"](s["logits"], history=s["history"], n_history=s["n_history"], n_prompt=s["n_prompt"],
                            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                            bias_off=s["bias_off"], bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"],
                            mask_row=s["mask_row"])
    return _process(s)


def _rms_rope(x, w, cs):
    """Norm of each head's 128 values (w None: none), then the rotation of the pairs (j, j + 64)."""
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    a, b = x[..., :HD // 2], x[..., HD // 2:]
    c, d = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat((a * c - b * d, b * c + a * d), -1)


def _exponent(amax):
    """The least e in E_MIN..E_MAX with amax <= 448 * 2^e: exact, from the parts of the number."""
    m, x = torch.frexp(amax)                                   # amax = m * 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _two(e):
    """2^e for whole e in -126..127, exact: the exponent's bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _scale(b):
    """2^(byte - 127), from the scales' bytes."""
    return _two(b.int() - 127)


def _codes(x):
    """Rounded to e4m3, the nearest value, ties to even."""
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _append(s):
    nq, nkv, page, block = s["nq"], s["nkv"], s["page"], s["block"]
    m, per = s["qkv"].shape[0], page // block
    off, ctx = s["q_off"].long(), s["ctx"].long()
    count = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(len(ctx), device="cuda"), count, output_size=m)
    past = (ctx - count)[seq]
    pos = past + torch.arange(m, device="cuda") - off[seq]
    x = s["qkv"].float().view(m, nq + 2 * nkv, HD)
    cs = s["rope"][pos]
    q = _rms_rope(x[:, :nq], s["q_norm"], cs)
    k = _rms_rope(x[:, nq:nq + nkv], s["k_norm"], cs)
    # the block of each token in the pool, and how many of the block's tokens were there before
    at = s["table"][seq, pos // page].long() * per + pos % page // block
    old = (past - pos // block * block).clamp(0, block)
    touched, back = torch.unique(at, return_inverse=True)
    there = torch.zeros_like(touched).index_reduce_(0, back, old, "amax")
    slot = torch.arange(block, device="cuda")
    for name, new in (("k", k), ("v", x[:, nq + nkv:])):
        codes = s[name + "_pages"].view(torch.uint8).view(-1, nkv, per, block, HD)
        scale = s[name + "_scale"].view(torch.uint8).view(-1, nkv, per)
        pg, sub = touched // per, touched % per
        was = scale[pg, :, sub].int() - 127
        top = torch.zeros(len(touched), nkv, device="cuda").index_reduce_(0, back, new.abs().amax(-1), "amax")
        e = torch.maximum(_exponent(top), torch.where(there[:, None] > 0, was, E_MIN))
        mine = codes[pg, :, sub]                                 # [blocks, nkv, block, 128]
        moved = _codes(mine.view(torch.float8_e4m3fn).float() * _two((was - e).clamp(min=-126))[..., None, None])
        mine = torch.where((slot < there[:, None])[:, None, :, None], moved.view(torch.uint8), mine)
        mine[back, :, pos % block] = _codes(new * _two(-e)[back][..., None]).view(torch.uint8)
        codes[pg, :, sub] = mine
        scale[pg, :, sub] = (e + 127).to(torch.uint8)
    return q.to(s["qkv"].dtype)


def _read(codes, scale, pages, block):
    """The values of pages; a code's four bits and a power of two are exact in bf16."""
    at = pages.long()
    x = codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    f = _scale(scale.view(torch.uint8)[at]).repeat_interleave(block, -1)
    return (x * f[..., None]).to(torch.bfloat16)


def _attend(s):
    nq, nkv, page = s["nq"], s["nkv"], s["page"]
    b, t, n = s["ctx"].shape[0], s["max_q"], s["max_ctx"]
    off, ctx = s["q_off"].long(), s["ctx"].long()
    count = off[1:] - off[:-1]
    j = torch.arange(n, device="cuda")
    # keys and values of each sequence side by side, [b, n, nkv, 128]
    at = s["table"][:, j // page].long()

    def side(name):
        x = s[name + "_pages"].view(torch.uint8)[at, :, j % page].view(torch.float8_e4m3fn).float()
        return x.mul_(_scale(s[name + "_scale"].view(torch.uint8)[at, :, j % page // s["block"]])[..., None])
    k, v = side("k"), side("v")
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


def _process(s):
    x = s["logits"].float()
    n, v = x.shape
    if s["history"] is not None:
        h = s["history"].long()
        j = torch.arange(h.shape[1], device="cuda")[None]
        inside = j < s["n_history"][:, None]
        said = inside & (j >= s["n_prompt"][:, None])
        every = torch.zeros_like(x).scatter_add_(1, h, inside.float())
        count = torch.zeros_like(x).scatter_add_(1, h, said.float())
        rep = s["repetition"][:, None]
        x = torch.where(every > 0, torch.where(x < 0, x * rep, x / rep), x)
        x = torch.where(count > 0, x - (s["presence"][:, None] + s["frequency"][:, None] * count), x)
    if s["bias"] is not None:
        off = s["bias_off"].long()
        row = torch.repeat_interleave(torch.arange(n, device="cuda"), off[1:] - off[:-1], output_size=len(s["bias"]))
        x = x.index_put((row, s["bias_ids"].long()), s["bias"], accumulate=True)
    if s["mask"] is not None:
        i = torch.arange(v, device="cuda")
        allowed = (s["mask"][:, i // 32] >> (i % 32).int()) & 1 != 0
        if s["mask_row"] is not None:
            allowed = allowed[s["mask_row"].clamp(min=0).long()] | (s["mask_row"] < 0)[:, None]
        x = x.masked_fill(~allowed, float("-inf"))
    return x.to(s["logits"].dtype)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "append8":
        return _exact_append(case, s)
    if case["op"] == "attend8":
        return _exact_attend(case, s)
    return _exact_process(case, s)


def _power(e):
    """2^e in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values(codes, scale, block):
    """Pages in 64 bits, [pages, nkv, page, 128]."""
    pages, nkv, page, _ = codes.shape
    f = _power(scale.view(torch.uint8).int() - 127)
    return (codes.double().view(pages, nkv, page // block, block, HD) * f[..., None, None]).view(codes.shape)


def _nearest(x, e):
    """x rounded to a step of e4m3 with the scale 2^e: three bits behind the leading one, 2^-9 at least."""
    y = x * _power(-e)
    step = torch.clamp(torch.frexp(y)[1] - 1, min=-6) - 3
    return (y * _power(-step)).round() * _power(step) * _power(e)


def _exact_append(case, s):
    nq, nkv, page, block = case["nq"], case["nkv"], case["page"], case["block"]
    x = s["qkv"].double().reshape(-1, nq + 2 * nkv, HD)
    lens = _lengths(case)
    pos = torch.cat([torch.arange(p, p + q, device="cuda") for q, p in lens])
    cos, sin = s["rope"].double()[pos].unbind(-1)

    def turned(h, w):
        if w is not None:
            h = h * (h.square().sum(-1, keepdim=True) / HD + 1e-6).rsqrt() * w.double()
        z = torch.complex(h[..., :64].contiguous(), h[..., 64:].contiguous()) * torch.complex(cos, sin)[:, None]
        return torch.cat((z.real, z.imag), -1)
    out = {"q": turned(x[:, :nq], s["q_norm"]).reshape(-1, nq, HD)}
    written = _written(case)
    for name, new in (("k", turned(x[:, nq:nq + nkv], s["k_norm"])), ("v", x[:, nq + nkv:])):
        # the pages written: old values, new values unrounded beside them, and which place holds which
        held = _values(s[name + "_pages"][s["pages"].long()], s[name + "_scale"].view(torch.uint8)[s["pages"].long()], block)
        was = s[name + "_scale"].view(torch.uint8)[s["pages"].long()].int() - 127          # [pages, nkv, blocks]
        fresh, kind = torch.zeros_like(held), torch.zeros(len(written), page, dtype=torch.int8, device="cuda")
        first = [0]
        for q, _ in lens:
            first.append(first[-1] + q)
        for i, (seq, j) in enumerate(written):
            q, p = lens[seq]
            a, b = max(p, j * page), min(q + p, (j + 1) * page)
            fresh[i, :, a - j * page:b - j * page] = new[first[seq] + a - p:first[seq] + b - p].transpose(0, 1)
            kind[i, :a - j * page] = 1
            kind[i, a - j * page:b - j * page] = 2
        kind = kind.view(len(written), 1, page // block, block)
        size = fresh.abs().amax(-1).view(len(written), nkv, page // block, block).amax(-1)
        e = torch.full_like(was, E_MIN)
        for t in range(E_MIN, 0):                         # the least exponent, found by trying them
            e = torch.where(size > 448 * 2.0 ** t, t + 1, e)
        e = torch.where((kind == 1).any(-1), torch.maximum(e, was), e)
        e = torch.where((kind == 2).any(-1), e, was)      # a block without new tokens stays as it is
        deep = e[..., None, None].expand(-1, -1, -1, block, HD)
        by_block = lambda t: t.view(len(written), nkv, page // block, block, HD)  # noqa: E731
        old, changed = by_block(held), _nearest(by_block(held), deep)
        got = torch.where((kind == 2)[..., None], _nearest(by_block(fresh), deep), torch.where((kind == 1)[..., None], changed, old))
        # behind the last token the codes stay, and the scale of a block with new tokens says what they stand for
        code = by_block(s[name + "_pages"][s["pages"].long()].double())
        got = torch.where(((kind == 0) & (kind == 2).any(-1, keepdim=True))[..., None], code * _power(deep), got)
        out[name] = got.reshape(held.shape)
    return out


def _exact_attend(case, s):
    nq, nkv, block = case["nq"], case["nkv"], case["block"]
    out, first = [], 0
    for i, (q, p) in enumerate(_lengths(case)):
        if not q:
            continue
        n = q + p
        pages = s["table"][i, :-(-n // case["page"])].long()
        k, v = (_values(s[c + "_pages"].view(torch.uint8)[pages].view(torch.float8_e4m3fn),
                        s[c + "_scale"].view(torch.uint8)[pages], block).transpose(1, 2).reshape(-1, nkv, HD)[:n]
                for c in "kv")
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


def _exact_process(case, s):
    import numpy as np
    x = s["logits"].double().cpu().numpy()
    host = {k: t.cpu().numpy() for k, t in s.items() if isinstance(t, torch.Tensor) and k != "logits"}
    v = x.shape[1]
    for i, row in enumerate(x):
        if "history" in host:
            ids = host["history"][i, :host["n_history"][i]]
            seen = np.unique(ids)
            rep = float(host["repetition"][i])
            row[seen] = np.where(row[seen] < 0, row[seen] * rep, row[seen] / rep)
            said, times = np.unique(ids[host["n_prompt"][i]:], return_counts=True)
            row[said] -= float(host["presence"][i]) + float(host["frequency"][i]) * times
        if "bias" in host:
            part = slice(host["bias_off"][i], host["bias_off"][i + 1])
            np.add.at(row, host["bias_ids"][part], host["bias"][part].astype(np.float64))
        if "mask" in host:
            m = i if "mask_row" not in host else host["mask_row"][i]
            if m >= 0:
                bits = np.unpackbits(host["mask"][m].view(np.uint8), bitorder="little")[:v]
                row[bits == 0] = -np.inf
    return torch.from_numpy(x)
