"""The bits that paged attention keeps of fp32 activations and pages, on inputs that show each of them.

Values have one nonzero place each (key j: place j), so that an output is one weight times one value and errors of
different weights cannot cancel; queries and keys have one or two, so that a score is one or two products.
"weights": scores within 1/2, so that little but the weights' own bits is left to be wrong.  "scores": two products
of about 64 that cancel to about 1, so that bits lost of a query or key are magnified 64 times.  A test on the CPU
shows that the bound is passed as soon as a part of an operand is lost."""
import math

import pytest

torch = pytest.importorskip("torch")

HD, PAGE, NKV = 128, 16, 4
U = 2.0 ** -24                       # half a step of fp32
LENS = [(2, 8), (1, 8), (2, 5), (2, 2)]
MANY = [(12, 12), (7, 8), (12, 12), (1, 8)]


def inputs(kind, lens, group, kv):
    """(q [m, heads, 128], k and v of each sequence [n, NKV, 128]) on the CPU, values of the type given."""
    g = torch.Generator().manual_seed(len(lens) * 7 + group + (kind == "scores"))

    def rand(*shape):
        return torch.rand(*shape, generator=g, dtype=torch.float64)
    m = sum(n for n, _ in lens)
    q = torch.zeros(m, NKV, group, HD, dtype=torch.float64)
    d0, d1 = [3, 17, 64, 5], [90, 18, 127, 4]
    ks, vs = [], []
    for h in range(NKV):
        if kind == "weights":
            q[:, h, :, d0[h]] = 0.25 + 0.25 * rand(m, group)
        else:
            a = 32 + 32 * rand(m, group)
            q[:, h, :, d0[h]] = a
            q[:, h, :, d1[h]] = a * (1 + (rand(m, group) - 0.5) * 2.0 ** -5)
    for _, n in lens:
        k, v = torch.zeros(n, NKV, HD, dtype=torch.float64), torch.zeros(n, NKV, HD, dtype=torch.float64)
        for h in range(NKV):
            x = 0.5 + 0.5 * rand(n)
            if kind == "weights":
                k[:, h, d0[h]] = 2 * rand(n) - 1
            else:
                if kv == torch.bfloat16:
                    x = x.to(kv).double()
                    y = x + torch.randint(-2, 3, (n,), generator=g) * 2.0 ** -8
                else:
                    x = x.float().double()
                    y = x + (rand(n) - 0.5) * 2.0 ** -6
                k[:, h, d0[h]], k[:, h, d1[h]] = x, -y
            v[torch.arange(n), h, torch.arange(n)] = 0.5 + 0.5 * rand(n)
        ks.append(k.to(kv))
        vs.append(v.to(kv))
    return q.float().reshape(m, NKV * group, HD), ks, vs


def cut(x, parts):
    """x as the sum of so many bf16 parts."""
    total, rest = torch.zeros_like(x, dtype=torch.float64), x.double()
    for _ in range(parts):
        p = rest.float().to(torch.bfloat16).double()
        total, rest = total + p, rest - p
    return total


def attend(q, ks, vs, lens, group, q_parts=0, p_parts=0, k_parts=0, v_parts=0):
    """Outputs in 64 bits (scale 1), with operands cut to so many parts (0: not at all), and what the bound needs."""
    out, size, spread, row = [], 0.0, 0.0, 0
    for (new, n), k, v in zip(lens, ks, vs):
        x = q[row:row + new].double().reshape(new, NKV, group, HD)
        row += new
        x, k, v = (cut(a, p) if p else a.double() for a, p in ((x, q_parts), (k, k_parts), (v, v_parts)))
        size = max(size, float(x.abs().max() * k.abs().max()))
        s = torch.einsum("thgd,nhd->thgn", x, k)
        hidden = torch.arange(n)[None] > (n - new + torch.arange(new))[:, None]
        spread = max(spread, float(s.abs().max()))
        s = s.masked_fill(hidden[:, None, None], -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        total = p.sum(-1, keepdim=True)
        if p_parts:
            p = cut(p.float(), p_parts)
        out.append(torch.einsum("thgn,nhd->thgd", p / total, v).reshape(new, NKV * group, HD))
    return torch.cat(out), size, spread


def relative_bound(size, spread, lens, p_bits):
    """Of an output, relative.  A score: each of at most four cuts of its terms to 24 bits costs 2^-23 of the largest
    product (the parts of q are exact).  The exponent: the factor (two roundings) and two more roundings, of at most 2
    and 3 times the largest score.  exp2: 2^-22 by its documentation, once for the weight and once where warps or CTAs
    are joined, and two roundings.  All of it once for the weight and once for their sum; the sum's additions; eight
    roundings on the way out; and p_bits for what the second product keeps of a weight."""
    n = max(c for _, c in lens)
    return 2 * (2.0 ** -21 * size + 7 * spread * U + 2.0 ** -21 + 2 * U) + (n + 8) * U + p_bits


# (kind, what is lost, bits of the weights that the path keeps): each of these has to pass the bound
LOST = [("weights", dict(p_parts=2), 0.0), ("weights", dict(p_parts=1), 2.0 ** -17), ("weights", dict(v_parts=2), 0.0),
        ("scores", dict(q_parts=2), 0.0), ("scores", dict(q_parts=2), 2.0 ** -17), ("scores", dict(k_parts=2), 0.0)]


@pytest.mark.parametrize("kind,lost,p_bits", LOST)
@pytest.mark.parametrize("lens,group", [(LENS, 4), (MANY, 1), (MANY, 4)])
def test_a_lost_part_passes_the_bound(lens, group, kind, lost, p_bits):
    kv = torch.float32 if "k_parts" in lost or "v_parts" in lost else torch.bfloat16
    q, k, v = inputs(kind, lens, group, kv)
    want, size, spread = attend(q, k, v, lens, group)
    less = attend(q, k, v, lens, group, **lost)[0]
    bound = relative_bound(size, spread, lens, p_bits)
    assert ((less - want).abs() > bound * want.abs()).any()
    whole = attend(q, k, v, lens, group, q_parts=3, p_parts=3, k_parts=3, v_parts=3)[0]
    assert ((whole - want).abs() <= 0.1 * bound * want.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["weights", "scores"])
@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,group", [(LENS, 4), (LENS, 1), (MANY, 1), (MANY, 4)])
def test_bits_of_fp32_activations(lens, group, kv, kind):
    """Few rows keep 24 bits of every operand, and so do fp32 pages; chunks over bf16 pages 17 of the weights."""
    import speech_lm_decode_gb300 as q3
    q, ks, vs = inputs(kind, lens, group, kv)
    pages = sum(-(-n // PAGE) for _, n in lens)
    k = torch.full((pages, NKV, PAGE, HD), float("nan"), dtype=kv)
    v = k.clone()
    table = torch.zeros(len(lens), 1, dtype=torch.int32)
    for i, (_, n) in enumerate(lens):
        table[i, 0] = pages - 1 - i
        k[pages - 1 - i, :, :n], v[pages - 1 - i, :, :n] = ks[i].transpose(0, 1), vs[i].transpose(0, 1)
    off = [0]
    for new, _ in lens:
        off.append(off[-1] + new)
    most = max(new for new, _ in lens)
    cache = q3.PagedKV(k.cuda(), v.cuda(), table.cuda(), n_q_heads=NKV * group)
    got = cache.attend(q.cuda(), torch.tensor(off, dtype=torch.int32).cuda(),
                       torch.tensor([n for _, n in lens], dtype=torch.int32).cuda(), most, scale=1.0).cpu().double()
    cache.check()
    want, size, spread = attend(q, ks, vs, lens, group)
    chunk = kv == torch.bfloat16 and most * group > 8
    bound = relative_bound(size, spread, lens, 2.0 ** -17 if chunk else 0.0)
    worst = ((got - want).abs() / want.abs().clamp(min=1e-30)).max()
    assert worst <= bound, (float(worst), bound)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float32])
def test_a_prompt_in_one_pass_and_in_chunks(kv):
    """The same prompts attended at once, in two chunks and token by token."""
    from paged_ref import attend64, make
    import speech_lm_decode_gb300 as q3
    lens = [(60, 60), (33, 33), (47, 47)]
    s = make(lens, 8, 4, PAGE, torch.float32, kv, seed=50)
    cache = q3.PagedKV(s["k"], s["v"], s["table"], n_q_heads=8)
    whole = cache.attend(s["q"], s["off"], s["ctx"], 60)
    want, bound = attend64(s)
    assert ((whole.double() - want).abs() <= bound).all()
    first = [int(o) for o in s["off"][:3]]
    for step in (25, 1):
        parts = torch.empty_like(whole)
        done = [0, 0, 0]
        while any(d < n for d, (n, _) in zip(done, lens)):
            now = [min(step, n - d) for d, (n, _) in zip(done, lens)]
            rows = torch.cat([torch.arange(f + d, f + d + c) for f, d, c in zip(first, done, now)]).cuda()
            done = [d + c for d, c in zip(done, now)]
            off = torch.tensor([0, now[0], now[0] + now[1], sum(now)], dtype=torch.int32, device="cuda")
            parts[rows] = cache.attend(s["q"][rows], off, torch.tensor(done, dtype=torch.int32, device="cuda"), step)
        cache.check()
        assert ((parts.double() - want).abs() <= bound).all(), step
        # against each other: both within fp32 sums of at most 60 terms and the weights' 17 bits
        diff, size = (parts.double() - whole.double()).square().mean().sqrt(), want.square().mean().sqrt()
        assert diff <= 2 * (2.0 ** -17 + 60 * U) * size, (step, float(diff / size))


def between(want, bound):
    """The bf16 values that a result within `bound` of want (relative) can round to: the least and the largest."""
    return tuple((want * (1 + s * bound)).float().to(torch.bfloat16).double() for s in (-1, 1))


BF16_LENS = [(LENS, 4), (LENS, 1), ([(5, 8), (3, 8), (5, 5)], 2)]


@pytest.mark.parametrize("lens,group", BF16_LENS)
def test_weights_in_bf16_pass_the_bound(lens, group):
    q, k, v = inputs("weights", lens, group, torch.bfloat16)
    q = q.to(torch.bfloat16).float()
    want, size, spread = attend(q, k, v, lens, group)
    lo, hi = between(want, relative_bound(size, spread, lens, 2.0 ** -17))
    for parts, inside in ((1, False), (2, True)):
        got = attend(q, k, v, lens, group, p_parts=parts)[0].float().to(torch.bfloat16).double()
        assert bool(((got >= lo) & (got <= hi)).all()) is inside


@pytest.mark.gpu
@pytest.mark.parametrize("lens,group", BF16_LENS)
def test_few_rows_of_bf16_activations_round_once(lens, group):
    """Their weights keep 17 bits, so that an output is what the fp32 result rounds to."""
    import speech_lm_decode_gb300 as q3
    q, ks, vs = inputs("weights", lens, group, torch.bfloat16)
    q = q.to(torch.bfloat16)
    pages = len(lens)
    k = torch.zeros(pages, NKV, PAGE, HD, dtype=torch.bfloat16)
    v = k.clone()
    for i, (_, n) in enumerate(lens):
        k[i, :, :n], v[i, :, :n] = ks[i].transpose(0, 1), vs[i].transpose(0, 1)
    off = [0]
    for new, _ in lens:
        off.append(off[-1] + new)
    cache = q3.PagedKV(k.cuda(), v.cuda(), torch.arange(pages, dtype=torch.int32)[:, None].cuda(), n_q_heads=NKV * group)
    got = cache.attend(q.cuda(), torch.tensor(off, dtype=torch.int32).cuda(),
                       torch.tensor([n for _, n in lens], dtype=torch.int32).cuda(), max(n for n, _ in lens),
                       scale=1.0).cpu().double()
    cache.check()
    want, size, spread = attend(q.float(), ks, vs, lens, group)
    lo, hi = between(want, relative_bound(size, spread, lens, 2.0 ** -17))
    assert ((got >= lo) & (got <= hi)).all()
