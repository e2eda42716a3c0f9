"""The paged cache in 8 bits: append (norms, rotation, blocks and their scales), attention over it and reading it back,
against 64-bit forms; run together, in graphs and on other streams; and what they refuse."""
import math

import pytest

torch = pytest.importorskip("torch")

from paged8_ref import (HD, HALF, attend64, cache_of, check_append, gather, make, nearest, need, power,  # noqa: E402
                        turned64, values)

pytestmark = pytest.mark.gpu
ACTS = {"bf16": torch.bfloat16, "f32": torch.float32}


def close(got, want, bound, what=""):
    err = (got.double() - want).abs()
    assert not torch.isnan(got).any(), what
    over = err > bound + 1e-30
    assert not over.any(), (what, float((err / (bound + 1e-30)).max()), torch.nonzero(over)[:4].tolist())


def rope_table(rows):
    ang = torch.arange(rows, device="cuda").double()[:, None] * 1e4 ** (-torch.arange(64, device="cuda").double() / 64)
    return torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()


def norms(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.2 * torch.randn(HD, generator=g, device="cuda") for _ in range(2))


def pools(s):
    return {n: s[n].view(torch.uint8).clone() for n in ("k", "ks", "v", "vs")}


# ---------------------------------------------------------------- append
# (sequences' (new, context)), q heads, kv heads, page, block
APPENDS = {
    "one": ([(1, 1)], 16, 8, 16, 16),
    "tokens": ([(1, 228), (1, 64), (1, 65), (1, 1), (1, 511), (1, 16), (1, 17)], 16, 8, 16, 16),
    "few": ([(4, 100), (3, 3), (1, 50), (2, 257), (0, 40), (4, 1029), (17, 40)], 16, 8, 32, 16),
    "prompts": ([(64, 64), (100, 100), (1, 77), (129, 300), (15, 31), (33, 33)], 16, 8, 32, 32),
    "blocks-of-64": ([(64, 64), (100, 130), (1, 77), (200, 300), (1, 129)], 16, 4, 128, 64),
    "one-block-a-page": ([(600, 700), (1, 1024), (30, 1050)], 4, 2, 1024, 1024),
    "heads-28-4": ([(19, 50), (1, 3)], 28, 4, 16, 16),
    "heads-16-1": ([(40, 90), (1, 3)], 16, 1, 64, 16),
    "heads-3-3": ([(40, 90), (5, 5), (0, 0)], 3, 3, 16, 16),
    "negative": ([(70, 40), (20, 1), (9, 0), (5, 5)], 16, 8, 16, 16),
    "many": ([((i * 7) % 5, max((i * 7) % 5, 3 + (i * 13) % 60)) for i in range(700)], 2, 1, 16, 16),
}


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", APPENDS)
def test_append_matches_64_bits(shape, act, norm):
    lens, nq, nkv, page, block = APPENDS[shape]
    s = make(lens, nq, nkv, page, block, ACTS[act], seed=len(shape), at_new=True)
    rows, width = int(s["off"][-1]), (nq + 2 * nkv) * HD
    g = torch.Generator(device="cuda").manual_seed(7)
    qkv = (torch.randn(rows + 2, width + 8, generator=g, device="cuda") * 1.5).to(ACTS[act])[:, :-8]   # strided rows
    rope = rope_table(max(c for _, c in lens) + 1)
    qn, kn = norms(3) if norm else (None, None)
    before, out = pools(s), torch.full((rows + 2, nq, HD), 3.0, dtype=ACTS[act], device="cuda")
    cache = cache_of(s)
    most = max(n for n, _ in lens)
    cache.append(qkv, s["off"], s["ctx"], most, rope, qn, kn, out=out)
    cache.check()
    q, qb, live = check_append(s, before, qkv, rope, qn, kn)
    close(out[:rows][live], q[live], (qb + q.abs() * HALF[ACTS[act]])[live], "q")
    assert (out[:rows][~live] == 3.0).all() and (out[rows:] == 3.0).all()
    # once more, the queries over the q columns: the same bits, as the blocks have their scales already
    now = pools(s)
    again = qkv.clone()
    cache.append(again, s["off"], s["ctx"], most, rope, qn, kn, out=again[:, :nq * HD])
    cache.check()
    assert torch.equal(again[:rows, :nq * HD].reshape(rows, nq, HD)[live], out[:rows][live])
    assert torch.equal(again[rows:], qkv[rows:]) and torch.equal(again[:, nq * HD:], qkv[:, nq * HD:])
    assert all(torch.equal(a, b) for a, b in zip(now.values(), pools(s).values()))


@pytest.mark.parametrize("block", [16, 32])
def test_token_by_token(block):
    """Blocks that grow while they fill: every step against the state before it."""
    nq, nkv, page = 4, 2, 32
    s = make([(1, 70), (1, 70)], nq, nkv, page, block, torch.float32, seed=5, at_new=True)
    s["ks"].fill_(200)         # a block's scale from an earlier owner: it does not count
    s["vs"].fill_(255)
    rope = rope_table(80)
    cache = cache_of(s)
    g = torch.Generator(device="cuda").manual_seed(8)
    for p in range(60):
        size = 2.0 ** (p % 13 if p < 30 else -(p % 7))
        qkv = torch.randn(2, (nq + 2 * nkv) * HD, generator=g, device="cuda") * size
        if p == 0:             # the second sequence starts with three tokens
            s["lens"], first = [(0, 0), (3, 3)], torch.randn(3, qkv.shape[1], generator=g, device="cuda")
            off, ctx = (torch.tensor(t, dtype=torch.int32).cuda() for t in ([0, 0, 3], [0, 3]))
            before = pools(s)
            cache.append(first, off, ctx, 3, rope)
            check_append({**s, "off": off}, before, first, rope, None, None)
        s["lens"] = [(1, p + 1), (1, p + 4)]
        s["ctx"].copy_(torch.tensor([c for _, c in s["lens"]], dtype=torch.int32))
        before = pools(s)
        cache.append(qkv, s["off"], s["ctx"], 1, rope)
        cache.check()
        check_append(s, before, qkv, rope, None, None)


@pytest.mark.parametrize("act", ACTS)
def test_values_at_the_ends_of_the_range(act):
    """Zeros, the least and the largest values, infinities and NaN: each in a block of its own, and in one that fills."""
    nq, nkv, page, block = 2, 1, 16, 16
    rows = [torch.zeros(HD), torch.full((HD,), 1e-38), torch.full((HD,), 2.0 ** -100 * 448), torch.full((HD,), 2.0 ** -100 * 449.0),
            torch.full((HD,), 448.0), torch.full((HD,), 450.0), torch.linspace(-448, 448, HD), torch.full((HD,), 2.0 ** 127 * 1.9),
            torch.full((HD,), float("inf")), torch.full((HD,), float("nan")), torch.linspace(-20, 20, HD), torch.full((HD,), -2.0 ** 120)]
    rows[10][5], rows[10][6], rows[10][7] = float("inf"), float("-inf"), float("nan")
    x = torch.stack(rows).cuda()
    for lens in ([(1, 1)] * len(rows), [(len(rows), len(rows))]):
        s = make(lens, nq, nkv, page, block, ACTS[act], seed=2, at_new=True)
        qkv = torch.cat((torch.randn(len(rows), nq * HD, device="cuda"), x, x), 1).to(ACTS[act]).contiguous()
        rope = torch.zeros(64, 64, 2, device="cuda")
        rope[..., 0] = 1.0         # no turn
        cache = cache_of(s)
        cache.append(qkv, s["off"], s["ctx"], len(rows), rope)
        cache.check()
        v = qkv[:, -HD:].double()
        at = [int(s["table"][i, 0]) for i in range(len(lens))]
        if len(lens) == 1:
            got, e = values(s["v"], s["vs"], block)[at[0], 0, :len(rows)], s["vs"][at[0], 0].int().expand(len(rows)) - 127
        else:
            got, e = values(s["v"], s["vs"], block)[at, 0, 0], s["vs"][at, 0, 0].int() - 127
        want = torch.where(torch.isfinite(v), nearest(v.nan_to_num(0, 0, 0), e[:, None].expand_as(v)), float("nan"))
        assert torch.equal(got.nan_to_num(7e77), want.nan_to_num(7e77))
        if len(lens) > 1:
            assert torch.equal(e, need(v.abs().nan_to_num(0, 0, 0).amax(-1)))


@pytest.mark.parametrize("act", ACTS)
def test_append_reports_what_is_out_of_range(act):
    import speech_lm_decode_gb300 as q3
    lens = [(20, 40), (3, 30), (2, 33), (1, 9), (4, 50)]
    s = make(lens, 4, 2, 16, 16, ACTS[act], seed=9, at_new=True)
    rows = int(s["off"][-1])
    qkv = torch.randn(rows, 8 * HD, device="cuda").to(ACTS[act])
    rope = rope_table(47)                 # positions 47.. of the last sequence are past it
    s["table"][0, 2] = -1                 # positions 32..39 of the first sequence
    s["table"][1, 1] = s["k"].shape[0]    # position 27..29 of the second
    cache = cache_of(s)
    before, out = pools(s), torch.full((rows, 4, HD), 3.0, dtype=ACTS[act], device="cuda")
    cache.append(qkv, s["off"], s["ctx"], 20, rope, out=out)
    with pytest.raises(q3.Q3Error):
        cache.check()
    cache.check()
    s["table"][0, 2] = s["table"][1, 1] = 0
    skip = {(0, p) for p in range(32, 40)} | {(1, p) for p in range(27, 30)} | {(4, p) for p in range(47, 50)}
    q, qb, live = check_append(s, before, qkv, rope, None, None, skip=skip)
    close(out[live], q[live], (qb + q.abs() * HALF[ACTS[act]])[live], "q")
    assert (out[~live] == 3.0).all()
    # lengths and offsets: a sequence that is out of range is skipped, the others are not
    for off, ctx, most, there in (([0, 20, 23, 25, 26, 30], [40, 30, 33, 9, 1 << 20], 20, [0, 1, 2, 3]),
                                  ([0, 20, 23, 25, 26, 31], [40, 30, 33, 9, 50], 20, [0, 1, 2, 3]),
                                  ([0, 20, 23, 25, 24, 28], [40, 30, 33, 9, 50], 20, [0, 1, 2, 4]),
                                  ([0, 20, 23, 25, 26, 30], [40, -1, 33, 9, 50], 20, [0, 2, 3, 4]),
                                  ([0, 20, 23, 25, 26, 30], [40, 30, 33, 9, 50], 5, [1, 2, 3, 4]),
                                  ([-2 ** 31, 2 ** 31 - 1, 23, 25, 26, 30], [40, 30, 33, 9, 50], 20, [2, 3, 4])):
        t = make(lens, 4, 2, 16, 16, ACTS[act], seed=9, at_new=True)
        cache = cache_of(t)
        out = torch.full((rows, 4, HD), 3.0, dtype=ACTS[act], device="cuda")
        o = torch.tensor(off, dtype=torch.int32).cuda()
        cache.append(qkv, o, torch.tensor(ctx, dtype=torch.int32).cuda(), most, rope_table(60), out=out)
        with pytest.raises(q3.Q3Error):
            cache.check()
        alone = make(lens, 4, 2, 16, 16, ACTS[act], seed=9, at_new=True)
        ok, claims = torch.zeros(rows, dtype=torch.bool, device="cuda"), torch.zeros(rows, device="cuda")
        for i in there:
            n = off[i + 1] - off[i]
            o1 = torch.tensor([0] * (i + 1) + [n] * (len(lens) - i), dtype=torch.int32).cuda()
            ref = cache_of(alone).append(qkv[off[i]:off[i + 1]], o1, torch.tensor(ctx, dtype=torch.int32).clamp(0, 60).cuda(), n, rope_table(60))
            ok[off[i]:off[i + 1]] |= (out[off[i]:off[i + 1]] == ref).flatten(1).all(1)
            claims[off[i]:off[i + 1]] += 1
        # (offsets that go back give row 24 to two sequences: its heads are the one's or the other's)
        assert torch.equal(ok | (claims > 1), claims > 0) and (out[claims == 0] == 3.0).all()
        got, want = pools(t), pools(alone)
        assert all(torch.equal(got[x], want[x]) for x in got), (off, ctx, most)


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nkv,page,block,nhd", [(8, 16, 16, False), (3, 64, 32, True), (1, 1024, 1024, False)])
def test_read(nkv, page, block, nhd, dtype):
    import speech_lm_decode_gb300 as q3
    s = make([(1, 3 * page + 5), (1, 2 * page)], nkv, nkv, page, block, torch.float32, seed=4, nhd=nhd, spread=30.0)
    cache = cache_of(s)
    n = s["k"].shape[0]
    ids = torch.tensor([n - 1, 0, 2, 2, 1], dtype=torch.int32).cuda()
    k, v = cache.read(ids, dtype=dtype)
    cache.check()
    for got, name in ((k, "k"), (v, "v")):
        want = values(s[name].view(torch.uint8)[ids.long()], s[name + "s"][ids.long()], block)
        assert got.dtype == dtype and torch.equal(got.double().nan_to_num(7e77), want.nan_to_num(7e77))
    into = torch.full_like(k, 5.0)
    bad = torch.tensor([0, n, -1, 1, 1 << 30], dtype=torch.int32).cuda()
    k2, _ = cache.read(bad, dtype=dtype, k_out=into)
    with pytest.raises(q3.Q3Error):
        cache.check()
    assert k2 is into and (into[[1, 2, 4]] == 5.0).all()
    assert torch.equal(into[[0, 3]].nan_to_num(7e7), cache.read(bad[[0, 3]].contiguous(), dtype=dtype)[0].nan_to_num(7e7))
    cache.check()
    assert cache.read(ids[:0])[0].shape == (0, nkv, page, HD)


# ---------------------------------------------------------------- attention
SHAPES = {
    "one": ([(1, 1)], 16, 8, 16),
    "decode": ([(1, 228), (1, 64), (1, 65), (1, 1), (1, 511)], 16, 8, 16),
    "decode-group-1": ([(1, 130), (1, 17)], 8, 8, 32),
    "decode-group-8": ([(1, 1000), (1, 129), (1, 16)], 32, 4, 64),
    "decode-group-7": ([(1, 300), (1, 31)], 28, 4, 16),
    "decode-group-16": ([(1, 200), (1, 2500)], 16, 1, 128),
    "few-new": ([(4, 100), (3, 3), (1, 50), (2, 257), (0, 40), (4, 1029)], 16, 8, 16),
    "few-new-group-3": ([(5, 133), (2, 18)], 6, 2, 32),
    "eight-new": ([(8, 133), (2, 18), (7, 700)], 8, 4, 64),
    "empty": ([(0, 0), (2, 0), (1, 0), (0, 10), (3, 1)], 16, 8, 16),
    "prompts": ([(64, 64), (100, 100), (1, 77), (129, 300), (128, 128), (63, 1000)], 16, 8, 16),
    "prompts-group-1": ([(130, 200), (257, 257)], 4, 4, 32),
    "prompts-group-5": ([(77, 200), (150, 151)], 10, 2, 16),
    "prompts-group-8": ([(33, 640), (300, 300)], 16, 2, 64),
    "negative": ([(70, 40), (200, 1), (90, 90)], 16, 8, 16),
    "big-page": ([(200, 2049), (1, 1025), (17, 700)], 16, 8, 1024),
    "page-256": ([(150, 600), (260, 260)], 4, 2, 256),
    "long": ([(1, 20011), (1, 9)], 16, 8, 64),
    "long-chunk": ([(300, 9001)], 4, 2, 64),
}


@pytest.mark.parametrize("block", ["16", "page"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_attention_matches_64_bits(shape, act, block):
    lens, nq, nkv, page = SHAPES[shape]
    s = make(lens, nq, nkv, page, page if block == "page" else 16, ACTS[act], seed=len(shape), extra_rows=2, spread=3.0)
    cache = cache_of(s)
    rows, most = int(s["off"][-1]), max(q for q, _ in lens)
    out = torch.full((rows + 2, nq, HD), 7.0, dtype=ACTS[act], device="cuda")
    got = cache.attend(s["q"], s["off"], s["ctx"], most, out=out)
    cache.check()
    want, bound = attend64(s)
    close(got[:rows], want, bound, shape)
    # rows behind the last sequence are left as they were
    assert (out[rows:] == 7.0).all()
    # the same call again, on the same workspace: the same bits
    again = cache.attend(s["q"], s["off"], s["ctx"], most)
    assert torch.equal(again[:rows], got[:rows])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new", [1, 4, 70])
def test_strided_rows_and_pages(act, new):
    """q as columns of a wider buffer, out likewise, pages laid out [page, position, head, 128]."""
    s = make([(new, 333), (1, 40), (new, new)], 16, 8, 32, 16, ACTS[act], seed=3, nhd=True)
    n = s["q"].shape[0]
    wide = torch.randn(n, 32, HD, device="cuda").to(ACTS[act])
    wide[:, :16] = s["q"]
    dst = torch.zeros(n, 20, HD, dtype=ACTS[act], device="cuda")
    cache = cache_of(s)
    cache.attend(wide[:, :16], s["off"], s["ctx"], new, scale=0.2, out=dst[:, 4:])
    cache.check()
    want, bound = attend64(s, scale=0.2)
    close(dst[:, 4:], want, bound)
    assert (dst[:, :4] == 0).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new", [1, 3, 150])
def test_in_place(act, new):
    """The outputs over the queries, items cut between CTAs among them."""
    s = make([(new, 3000), (new, 400), (1, 77)], 16, 4, 16, 16, ACTS[act], seed=14)
    cache = cache_of(s)
    want = cache.attend(s["q"], s["off"], s["ctx"], new)
    q = s["q"].clone()
    got = cache.attend(q, s["off"], s["ctx"], new, out=q)
    cache.check()
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new,spread", [(1, 40.0), (4, 40.0), (1, 6.0), (70, 6.0)])
def test_scales_that_differ_widely(new, spread, act):
    """Few rows take any scales; many rows those within 2^12 of each other without a bit lost."""
    s = make([(new, 700), (new, 90), (1, 300)], 8, 4, 32, 16, ACTS[act], seed=42, spread=spread)
    cache = cache_of(s)
    # with keys of very unlike size a softmax follows the largest alone: small scores keep all of them in play
    scale = 2.0 ** (-spread - 4)
    got = cache.attend(s["q"], s["off"], s["ctx"], new, scale=scale)
    cache.check()
    want, bound = attend64(s, scale=scale)
    close(got, want, bound)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new", [1, 3, 40, 150])
@pytest.mark.parametrize("scale", [1e-38, 1.4e-45, 1e-30])
def test_scales_next_to_zero(scale, new, act):
    """Every score is the same then: the outputs are means of the values."""
    s = make([(new, 700), (new, 40), (1, 300)], 8, 4, 16, 16, ACTS[act], seed=42)
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], new, scale=scale)
    cache.check()
    want, bound = attend64(s, scale=scale)
    close(got, want, bound, str(scale))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_queries_of_any_size(size, new, act):
    """Rows of very unlike size, zeros among them; the scale makes up for it."""
    s = make([(new, 400), (new, 90)], 8, 4, 16, 16, ACTS[act], seed=41)
    s["q"] = (s["q"].float() * size).to(ACTS[act])
    s["q"][0, 1] = 0
    s["q"][0, 2, :64] *= 2.0 ** -12
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], new, scale=0.1 / size)
    cache.check()
    want, bound = attend64(s, scale=0.1 / size)
    close(got, want, bound, str(size))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new", [1, 64])
def test_growing_scores(act, new):
    """The running maximum moves at every tile, by a little and by a lot."""
    s = make([(new, 900), (new, 333)], 8, 4, 16, 16, ACTS[act], seed=17)
    g = torch.Generator(device="cuda").manual_seed(3)
    for i, (_, c) in enumerate(s["lens"]):
        for p in range(0, c, 16):
            s["ks"][int(s["table"][i, p // 16]), :, 0] = 127 - 7 + (p // 16 % 9) // 2
    s["q"] = (torch.rand(s["q"].shape, generator=g, device="cuda") + 0.5).to(ACTS[act])
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], new, scale=0.5)
    cache.check()
    want, bound = attend64(s, scale=0.5)
    close(got, want, bound)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("lens", [[(1, 700), (1, 90)], [(3, 700), (2, 90)], [(9, 5000)], [(150, 700), (40, 90)]])
def test_nan_stays_where_it_belongs(lens, act):
    """A NaN key gives NaN to the rows that see it, a NaN query to its own row; no other row changes."""
    s = make(lens, 8, 2, 16, 16, ACTS[act], seed=18)
    most = max(n for n, _ in lens)
    base = cache_of(s).attend(s["q"], s["off"], s["ctx"], most)
    n, c = lens[0]
    # the last key of sequence 0: its last token alone sees it
    page, slot = int(s["table"][0, (c - 1) // 16]), (c - 1) % 16
    codes = s["k"].view(torch.uint8)
    was = codes[page, 1, slot, 9].clone()
    codes[page, 1, slot, 9] = 0xff
    got = cache_of(s).attend(s["q"], s["off"], s["ctx"], most)
    row = int(s["off"][1]) - 1
    want = base.clone()
    want[row, 4:] = float("nan")
    assert torch.equal(got.nan_to_num(7e7), want.nan_to_num(7e7))
    codes[page, 1, slot, 9] = was
    s["q"][0, 3, 5] = float("nan")
    got = cache_of(s).attend(s["q"], s["off"], s["ctx"], most)
    want = base.clone()
    want[0, 3] = float("nan")
    assert torch.equal(got.nan_to_num(7e7), want.nan_to_num(7e7))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new", [2, 40])
def test_a_block_whose_scale_is_nan(new, act):
    """Its keys give NaN to the rows that see one of them, and to no other."""
    s = make([(new, 333), (new, 90)], 4, 2, 16, 16, ACTS[act], seed=19)
    base = cache_of(s).attend(s["q"], s["off"], s["ctx"], new)
    s["ks"][int(s["table"][0, 20]), 1] = 255         # positions 320..332 of sequence 0, head 1
    got = cache_of(s).attend(s["q"], s["off"], s["ctx"], new)
    last = 333 - new + torch.arange(new, device="cuda")
    want = base.clone()
    want[:new, 2:][last >= 320] = float("nan")
    assert torch.equal(got.nan_to_num(7e7), want.nan_to_num(7e7))


GONE = {"few": [(2, 700), (1, 90)], "chunk": [(90, 700), (40, 130)], "one-tile": [(40, 3000)]}


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("case", GONE)
def test_keys_of_pages_out_of_range_do_not_count(case, act, page):
    import speech_lm_decode_gb300 as q3
    lens = GONE[case]
    s = make(lens, 8, 4, page, 16, ACTS[act], seed=31)
    n = s["k"].shape[0]
    gone = [(0, 0), (0, 3), (0, 4)]
    keep = {}
    for (i, j), bad in zip(gone, (-1, n, -2 ** 31)):
        keep[i, j] = int(s["table"][i, j])
        s["table"][i, j] = bad
    most = max(q for q, _ in lens)
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], most)
    with pytest.raises(q3.Q3Error):
        cache.check()
    cache.check()
    for (i, j), was in keep.items():
        s["table"][i, j] = was
    want, bound = attend64(s)
    close(got[lens[0][0]:], want[lens[0][0]:], bound[lens[0][0]:])
    # sequence 0 again, its scores at those positions -inf
    nn, c = lens[0]
    k, v = gather(s, 0, c)
    dead = torch.zeros(c, dtype=torch.bool, device="cuda")
    for _, j in gone:
        dead[j * page:(j + 1) * page] = True
    last = c - nn + torch.arange(nn, device="cuda")
    hide = dead[None] | (torch.arange(c, device="cuda")[None] > last[:, None])
    for h in range(8):
        x = (s["q"][:nn, h].double() @ k[:, h // 2].T * HD ** -0.5).masked_fill(hide, -math.inf)
        p = torch.softmax(x, -1).nan_to_num(0.0)
        o = p @ v[:, h // 2]
        b = (p @ v[:, h // 2].abs()) * 2.0 ** -9 + o.abs() * HALF[ACTS[act]] + 1e-30
        assert ((got[:nn, h].double() - o).abs() <= b).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new", [1, 70])
def test_offsets_and_lengths_out_of_range(act, new):
    import speech_lm_decode_gb300 as q3
    lens = [(new, 200), (1, 90), (new, 100)]
    s = make(lens, 8, 4, 16, 16, ACTS[act], seed=32)
    rows = int(s["off"][-1])
    base = cache_of(s).attend(s["q"], s["off"], s["ctx"], new)
    for off, most, there in (([0, new, new + 1, rows + 1], new, [0, 1]), ([0, new, 0, rows + 5], new, [0]),
                             ([-2 ** 31, 2 ** 31 - 1, new + 1, rows], new, [2]), ([0, new, new + 1, rows], 0, [])):
        out = torch.full_like(base, 9.0)
        cache = cache_of(s)
        cache.attend(s["q"], torch.tensor(off, dtype=torch.int32).cuda(), s["ctx"], most, out=out)
        if most:
            with pytest.raises(q3.Q3Error):
                cache.check()
        live = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for i in there:
            live[off[i]:off[i + 1]] = True
        assert torch.equal(out[live], base[live]) and (out[~live] == 9.0).all()
    # a context past the table or below zero is cut to it
    for ctx in (1 << 28, -5):
        c2 = s["ctx"].clone()
        c2[1] = ctx
        cache = cache_of(s)
        got = cache.attend(s["q"], s["off"], c2, new)
        with pytest.raises(q3.Q3Error):
            cache.check()
        live = torch.ones(rows, dtype=torch.bool, device="cuda")
        live[new] = False
        close(got[live], base[live].double(), base[live].double().abs() * 2.0 ** -6 + 1e-2)
        if ctx < 0:
            assert (got[new] == 0).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("most", [1, 3, 40])
def test_many_sequences(act, most):
    """More sequences than a CTA has threads, some without new tokens or without any."""
    g = torch.Generator().manual_seed(most)
    lens = [(int(torch.randint(0, most + 1, (1,), generator=g)), int(torch.randint(0, 60, (1,), generator=g)))
            for _ in range(1500)]
    s = make(lens, 2, 1, 16, 16, ACTS[act], seed=21)
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], most)
    cache.check()
    want, bound = attend64(s)
    close(got, want, bound)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("new", [1, 50])
def test_sequences_that_share_pages(act, new):
    s = make([(new, 300), (new, 333), (new, 290)], 8, 2, 16, 16, ACTS[act], seed=22)
    s["table"][1, :12] = s["table"][0, :12]
    s["table"][2, :15] = s["table"][0, :15]
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], new)
    cache.check()
    want, bound = attend64(s)
    close(got, want, bound)


def test_pages_past_32_bits():
    """A pool of more than 2^32 bytes, the sequence's pages at its end."""
    n_pages, page = 33000, 128
    codes = torch.zeros(n_pages, 8, page, HD, dtype=torch.uint8, device="cuda")
    scale = torch.full((n_pages, 8, page // 16), 120, dtype=torch.uint8, device="cuda")
    for new in (1, 80):
        s = make([(new, 300)], 16, 8, page, 16, torch.bfloat16, seed=23)
        last = torch.arange(n_pages - s["k"].shape[0], n_pages, device="cuda")
        big = {}
        for name in ("k", "v"):
            big[name], big[name + "s"] = codes.clone(), scale.clone()
            big[name][last], big[name + "s"][last] = s[name].view(torch.uint8), s[name + "s"]
            big[name] = big[name].view(torch.float8_e4m3fn)
        table = torch.where(s["table"] < 1 << 20, s["table"] + int(last[0]), s["table"]).to(torch.int32)
        t = {**s, **big, "table": table}
        cache = cache_of(t)
        got = cache.attend(s["q"], s["off"], s["ctx"], new)
        cache.check()
        assert torch.equal(got, cache_of(s).attend(s["q"], s["off"], s["ctx"], new))
        rope, qkv = rope_table(400), torch.randn(new, 32 * HD, device="cuda").to(torch.bfloat16)
        cache.append(qkv, s["off"], s["ctx"], new, rope)
        cache.check()
        cache_of(s).append(qkv, s["off"], s["ctx"], new, rope)
        for name in ("k", "v"):
            assert torch.equal(big[name].view(torch.uint8)[last], s[name].view(torch.uint8))
            assert torch.equal(big[name + "s"][last], s[name + "s"]) and not big[name].view(torch.uint8)[:int(last[0])].any()
        k, _ = cache.read(last.to(torch.int32))
        assert torch.equal(k.nan_to_num(7e7), cache_of(s).read(torch.arange(len(last), dtype=torch.int32, device="cuda"))[0].nan_to_num(7e7))
        del t, big, cache, k


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("lens", [[(1, 3000), (1, 700)], [(4, 3000), (3, 700)], [(150, 700), (200, 1500)]])
def test_bits_that_attention_keeps(lens, act):
    """Errors relative to the result's norm.  fp32: parts of 22 bits and sums of fp32, 5e-7 and less here; a part that is
    lost leaves 11 bits, 1e-4.  bf16: the output's rounding is 1.7e-3 of the norm (uniform within half a step of 2^-8,
    values uniform between two powers of two), weights of 11 bits add 1e-4 to it at most; of 8 bits they would make it 2.3e-3."""
    s = make(lens, 8, 4, 32, 16, ACTS[act], seed=71)
    got = cache_of(s).attend(s["q"], s["off"], s["ctx"], max(n for n, _ in lens))
    want, _ = attend64(s)
    off = float((got.double() - want).norm() / want.norm())
    assert off < (2e-6 if act == "f32" else 1.8e-3), off


def test_many_rows_of_fp32_over_a_long_context():
    """The tensor cores cut what they add, so that an output kept there falls behind by as much with every tile: 1.1e-5
    of the result after 120 tiles.  The eight tiles that it is kept for are 64 sums that lose a step of 2^-24 of it each
    at most, 3.8e-6."""
    s = make([(700, 15000)], 16, 8, 64, 64, torch.float32, seed=73)
    got = cache_of(s).attend(s["q"], s["off"], s["ctx"], 700)
    want, _ = attend64(s)
    off = float((got.double() - want).norm() / want.norm())
    assert off < 4e-6, off


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("lens", [[(150, 3000), (40, 333)], [(40, 900), (17, 64), (1, 500)]])
def test_a_wait_that_runs_out(lens, act):
    """Every CTA's wait for room for its n-th tile of codes counts as run out, at the start of an item or inside: the call
    returns, says so, and leaves counters with which the next call on the workspace gives the bits that it should."""
    import speech_lm_decode_gb300 as q3
    s = make(lens, 8, 4, 16, 16, ACTS[act], seed=44)
    most = max(q for q, _ in lens)
    cache = cache_of(s)
    want = cache.attend(s["q"], s["off"], s["ctx"], most)
    cache.check()
    (ws,) = cache._ws.values()
    for n in list(range(1, 14)) + [20, 33]:
        broken = cache_of(s, inject_timeout=n)
        broken.attend(s["q"], s["off"], s["ctx"], most)
        torch.cuda.synchronize()
        e = int(broken.err.item())
        assert e in (0, q3.Q3PAGED_ERR_TIMEOUT) and (e or n > 2)     # (a CTA may have fewer tiles than that)
        assert list(broken._ws.values())[0] is ws
        assert not ws[:q3.Q3PAGED_COUNTER_BYTES].any()
        assert torch.equal(cache.attend(s["q"], s["off"], s["ctx"], most), want)
        cache.check()


def test_scales_past_what_many_rows_keep():
    """Blocks whose scales are 2^30 apart: finite results, and those of the blocks that count."""
    for act in ACTS.values():
        s = make([(70, 200), (9, 90)], 4, 2, 16, 16, act, seed=72)
        s["ks"][int(s["table"][0, 3])] -= 30
        s["vs"][int(s["table"][0, 5])] -= 30
        got = cache_of(s).attend(s["q"], s["off"], s["ctx"], 70)
        want, bound = attend64(s)
        # what such a block loses is below 2^-24 of its neighbours' values
        k, v = gather(s, 0, 200)
        close(got, want, bound + float(v.abs().max()) * 2.0 ** -20)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("act", ACTS)
def test_prompt_then_tokens(act):
    """A prompt in one pass, then tokens one by one: append and attend in turn, each step's attention against 64 bits
    of what the cache holds then, in a graph that is replayed with new lengths; and the cache's error against
    unrounded keys and values: half a step of e4m3 or of its least one, twice where a block grew."""
    nq, nkv, page, block, T = 8, 4, 16, 16, ACTS[act]
    s = make([(37, 37), (5, 5)], nq, nkv, page, block, T, seed=51, spare=12, at_new=True)
    table = torch.arange(12, dtype=torch.int32).view(2, 6).cuda()
    s["table"] = table
    cache, rope = cache_of(s), rope_table(96)
    qn, kn = norms(5)
    g = torch.Generator(device="cuda").manual_seed(6)
    width = (nq + 2 * nkv) * HD
    qkv = torch.randn(42, width, generator=g, device="cuda").to(T)
    q = cache.append(qkv, s["off"], s["ctx"], 37, rope, qn, kn)
    o = cache.attend(q, s["off"], s["ctx"], 37)
    cache.check()
    s["q"] = q
    close(o, *attend64(s))
    step = torch.zeros(2, width, dtype=T, device="cuda")
    off, ctx = torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), torch.tensor([38, 6], dtype=torch.int32).cuda()
    every = [[qkv[:37]], [qkv[37:]]]
    kept = pools(s)
    cache.attend(cache.append(step, off, ctx, 1, rope, qn, kn), off, ctx, 1)
    for n, t in kept.items():
        s[n].view(torch.uint8).copy_(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq = cache.append(step, off, ctx, 1, rope, qn, kn)
        go = cache.attend(gq, off, ctx, 1)
    for i in range(40):
        step.copy_(torch.randn(2, width, generator=g, device="cuda").to(T))
        ctx.copy_(torch.tensor([38 + i, 6 + i], dtype=torch.int32))
        every[0].append(step[:1].clone())
        every[1].append(step[1:].clone())
        graph.replay()
        torch.cuda.synchronize()
        cache.check()
        t = {**s, "lens": [(1, 38 + i), (1, 6 + i)], "off": off, "ctx": ctx, "q": gq}
        close(go, *attend64(t), str(i))
    for i, n in ((0, 77), (1, 45)):
        x = torch.cat(every[i])
        assert x.shape[0] == n
        _, (k, kb), v = turned64(x, torch.arange(n, device="cuda"), rope, qn, kn, 1e-6, nq, nkv)
        for got, want, b, name in zip(gather(s, i, n), (k, v), (kb, 0), "kv"):
            f = power(s[name + "s"][table[i].long()].int() - 127).transpose(1, 2).reshape(-1, nkv)[:-(-n // 16)]
            f = f.repeat_interleave(16, 0)[:n, :, None]
            # (an entry that was rounded twice is off by two halves of a step; one below 2^-6 of the scale by 2^-10 of it)
            far = (got - want).abs() - b
            first = want.abs() * 2.0 ** -4 + f * 2.0 ** -10
            assert (far <= 2.2 * first).all()


def test_a_serving_step():
    """Append, attention, logits, penalties and mask, draw, the history grown on the device: steps of a captured graph
    against 64 bits and against the same steps eager."""
    import speech_lm_decode_gb300 as q3
    from paged8_ref import process64
    nq, nkv, n, vocab, T = 4, 2, 3, 1000, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(81)
    emb = torch.randn(vocab, (nq + 2 * nkv) * HD, generator=g, device="cuda").to(T)
    head = (torch.randn(nq * HD, vocab, generator=g, device="cuda") * 0.3).to(T)
    words = torch.randint(-2 ** 31, 2 ** 31, (2, 32), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    rope = rope_table(40)
    full = dict(temperature=torch.ones(n, device="cuda"), top_k=torch.full((n,), 20, dtype=torch.int32, device="cuda"),
                top_p=torch.full((n,), 0.9, device="cuda"), min_p=torch.zeros(n, device="cuda"))
    us = torch.rand(20, n, generator=g, device="cuda")

    def program():
        s = make([(1, 1)] * n, nq, nkv, 16, 16, T, seed=82, spare=9, at_new=True)
        s["table"] = torch.arange(9, dtype=torch.int32).view(3, 3).cuda()
        st = {"s": s, "cache": cache_of(s), "ctx": torch.ones(n, dtype=torch.int32, device="cuda"),
              "hist": torch.full((n, 40), -1, dtype=torch.int32, device="cuda"), "said": torch.zeros(n, dtype=torch.int32, device="cuda"),
              "ids": torch.arange(n, dtype=torch.int32, device="cuda"), "u": torch.zeros(n, device="cuda"),
              "off": torch.arange(n + 1, dtype=torch.int32, device="cuda")}
        kw = dict(history=st["hist"], n_history=st["said"], repetition=torch.full((n,), 1.3, device="cuda"),
                  presence=torch.full((n,), 0.4, device="cuda"), frequency=torch.full((n,), 0.2, device="cuda"),
                  mask=words, mask_row=torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda"))

        def step():
            qkv = emb[st["ids"].long()]
            q = st["cache"].append(qkv, st["off"], st["ctx"], 1, rope)
            o = st["cache"].attend(q, st["off"], st["ctx"], 1)
            raw = (o.view(n, -1) @ head).float()
            logits = q3.process_logits(raw, **kw)
            ids, logprob = q3.sample_given(logits, st["u"], **full)
            out = [t.clone() for t in (q, o, raw, logits, ids, logprob)]
            st["hist"].scatter_(1, st["said"].long()[:, None], ids[:, None])
            st["ids"].copy_(ids)
            st["said"] += 1
            st["ctx"] += 1
            return out
        return st, kw, step
    st, kw, step = program()
    st2, _, step2 = program()
    keep = {k: v.clone() for k, v in st2.items() if isinstance(v, torch.Tensor)}
    step2()
    for k, v in keep.items():
        st2[k].copy_(v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = step2()
    for i in range(20):
        for t in (st, st2):
            t["u"].copy_(us[i])
        said = {k: v.cpu().numpy().copy() for k, v in kw.items()}
        lens = [(1, i + 1)] * n
        q, o, raw, logits, ids, logprob = step()
        graph.replay()
        torch.cuda.synchronize()
        st["cache"].check()
        st2["cache"].check()
        assert all(torch.equal(a, b) for a, b in zip((q, o, raw, logits, ids, logprob), replayed)), i
        close(o, *attend64({**st["s"], "q": q, "lens": lens, "off": st["off"]}), str(i))
        want, bound = process64(raw.cpu().numpy(), **said)
        err = (logits.double().cpu() - torch.from_numpy(want)).abs()
        assert (err.nan_to_num(0) <= torch.from_numpy(bound) + torch.from_numpy(want).abs().nan_to_num(0, 0, 0) * 2.0 ** -24).all()
        for r, m in ((0, 0), (1, 1)):
            assert int(words[m, int(ids[r]) // 32]) >> (int(ids[r]) % 32) & 1


@pytest.mark.parametrize("act", ACTS)
def test_two_streams_at_once(act):
    states = [make([(1, 900), (1, 70)], 16, 8, 16, 16, ACTS[act], seed=61), make([(60, 900), (9, 70)], 8, 2, 16, 16, ACTS[act], seed=62)]
    want = [cache_of(s).attend(s["q"], s["off"], s["ctx"], max(n for n, _ in s["lens"])) for s in states]
    caches = [cache_of(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [[], []]
    for _ in range(20):
        for i, (st, s) in enumerate(zip(streams, states)):
            with torch.cuda.stream(st):
                got[i].append(caches[i].attend(s["q"], s["off"], s["ctx"], max(n for n, _ in s["lens"])))
    torch.cuda.synchronize()
    for i in range(2):
        caches[i].check()
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("new", [1, 60])
def test_two_graphs_side_by_side(new):
    s = make([(new, 900), (new, 700)], 16, 8, 16, 16, torch.bfloat16, seed=63)
    cache = cache_of(s)
    want = cache.attend(s["q"], s["off"], s["ctx"], new)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(cache.attend(s["q"], s["off"], s["ctx"], new))
        graphs.append(gr)
    side = torch.cuda.Stream()
    for _ in range(10):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        here = cache.attend(s["q"], s["off"], s["ctx"], new)
    torch.cuda.synchronize()
    cache.check()
    assert torch.equal(here, want) and all(torch.equal(o, want) for o in outs)


def test_one_workspace_for_both_kinds_of_cache():
    import speech_lm_decode_gb300 as q3
    from paged_ref import make as make16
    s8 = make([(1, 900), (1, 70)], 16, 8, 16, 16, torch.bfloat16, seed=64)
    s16 = make16([(1, 900), (1, 70)], 16, 8, 16, torch.bfloat16, torch.bfloat16, seed=64)
    c8, c16 = cache_of(s8), q3.PagedKV(s16["k"], s16["v"], s16["table"], n_q_heads=16)
    assert c8.ws_bytes == c16.ws_bytes
    want = [c.attend(s["q"], s["off"], s["ctx"], 1) for c, s in ((c8, s8), (c16, s16))]
    for _ in range(3):
        for c, s, w in ((c8, s8, want[0]), (c16, s16, want[1])):
            assert torch.equal(c.attend(s["q"], s["off"], s["ctx"], 1), w)
    assert list(c8._ws.values())[0] is list(c16._ws.values())[0]


def test_refusals():
    import speech_lm_decode_gb300 as q3
    s = make([(1, 40), (2, 9)], 16, 8, 32, 16, torch.bfloat16, seed=65)
    k, v, ks, vs, table = s["k"], s["v"], s["ks"], s["vs"], s["table"]

    def no(*a, error=ValueError, nq=16, **kw):
        with pytest.raises(error):
            q3.PagedKV8(*a, n_q_heads=nq, **kw)
    no(k.view(torch.uint8), v.view(torch.uint8), ks, vs, table)
    no(k.float(), v.float(), ks, vs, table)
    no(k, v[1:], ks, vs, table)
    no(k, v, ks.float(), vs, table)
    no(k, v, ks[:1], vs, table)
    no(k, v, ks, vs[..., :1], table)
    no(k, v, ks[..., :0], vs[..., :0], table)
    no(k, v, ks.transpose(0, 1).contiguous().transpose(0, 1), vs, table)
    no(k, v, ks.cpu(), vs, table)
    no(k, v, ks, vs, table.long())
    four = torch.zeros(k.shape[0], 8, 4, dtype=torch.uint8, device="cuda")
    no(k, v, four, four, table, error=q3.Q3Error)          # blocks of eight
    no(k, v, ks, vs, table, nq=12, error=q3.Q3Error)
    no(k, v, ks, vs, table, error=q3.Q3Error, inject_timeout=-1)
    with pytest.raises(ValueError):
        q3.PagedKV(k, v, table, n_q_heads=16)               # the other cache takes no codes
    cache = q3.PagedKV8(k, v, ks.view(torch.float8_e8m0fnu), vs.view(torch.float8_e8m0fnu), table, n_q_heads=16)
    q, off, ctx = s["q"], s["off"], s["ctx"]
    for bad in (dict(q=q.half()), dict(q=q[:, :8]), dict(q=q.cpu()), dict(off=off.long()), dict(off=off[:-1]), dict(ctx=ctx[:1]),
                dict(out=torch.empty(1, 16, HD, dtype=torch.bfloat16, device="cuda")), dict(out=torch.empty_like(q, dtype=torch.float32))):
        a = {**dict(q=q, off=off, ctx=ctx, out=None), **bad}
        with pytest.raises(ValueError):
            cache.attend(a["q"], a["off"], a["ctx"], 2, out=a["out"])
    for bad in (dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(q3.Q3Error):
            cache.attend(q, off, ctx, 2, **bad)
    qkv, rope = torch.randn(3, 32 * HD, device="cuda").to(torch.bfloat16), rope_table(64)
    w = torch.ones(HD, device="cuda")
    for bad in (dict(rope=rope.double()), dict(rope=rope[:, :32]), dict(q_norm=w.bfloat16(), k_norm=w), dict(qkv=qkv[:, :-128])):
        a = {**dict(qkv=qkv, rope=rope, q_norm=None, k_norm=None), **bad}
        with pytest.raises(ValueError):
            cache.append(a["qkv"], off, ctx, 2, a["rope"], a["q_norm"], a["k_norm"])
    with pytest.raises(q3.Q3Error):
        cache.append(qkv, off, ctx, 2, rope, q_norm=w)
    with pytest.raises(ValueError):
        cache.read(torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        cache.read(torch.zeros(2, dtype=torch.int32, device="cuda"), dtype=torch.float16)
    with pytest.raises(ValueError):
        cache.read(torch.zeros(2, dtype=torch.int32, device="cuda"), k_out=torch.empty(1, 8, 32, HD, device="cuda"))
    cache.check()
