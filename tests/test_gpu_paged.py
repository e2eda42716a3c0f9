"""The paged cache: append (norms, rotation, store) and attention over it, against 64-bit forms; run together, in
graphs and on other streams; and what they refuse."""
import pytest

torch = pytest.importorskip("torch")

from paged_ref import HD, HALF, append64, attend64, make  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"bf16": (torch.bfloat16, torch.bfloat16), "f32": (torch.float32, torch.bfloat16),
         "f32kv": (torch.float32, torch.float32)}


def cache_of(s):
    import speech_lm_decode_gb300 as q3
    return q3.PagedKV(s["k"], s["v"], s["table"], n_q_heads=s["nq"])


def close(got, want, bound, what=""):
    err = (got.double() - want).abs()
    assert not torch.isnan(got).any(), what
    over = err > bound + 1e-30
    assert not over.any(), (what, float((err / (bound + 1e-30)).max()), torch.nonzero(over)[:4].tolist())


# (sequences' (new, context)), q heads, kv heads, page
SHAPES = {
    "one": ([(1, 1)], 16, 8, 16),
    "decode": ([(1, 228), (1, 64), (1, 65), (1, 1), (1, 511)], 16, 8, 16),
    "decode-group-1": ([(1, 130), (1, 17)], 8, 8, 32),
    "decode-group-8": ([(1, 1000), (1, 129), (1, 16)], 32, 4, 64),
    "decode-group-7": ([(1, 300), (1, 31)], 28, 4, 16),
    "decode-group-16": ([(1, 200), (1, 2500)], 16, 1, 128),
    "few-new": ([(4, 100), (3, 3), (1, 50), (2, 257), (0, 40), (4, 1029)], 16, 8, 16),
    "few-new-group-3": ([(5, 133), (2, 18)], 6, 2, 32),
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


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_attention_matches_64_bits(shape, types):
    lens, nq, nkv, page = SHAPES[shape]
    act, kv = TYPES[types]
    s = make(lens, nq, nkv, page, act, kv, seed=len(shape), extra_rows=2)
    cache = cache_of(s)
    rows = int(s["off"][-1])
    out = torch.full((rows + 2, nq, HD), 7.0, dtype=act, device="cuda")
    got = cache.attend(s["q"], s["off"], s["ctx"], max(q for q, _ in lens), out=out)
    cache.check()
    want, bound = attend64(s)
    close(got[:rows], want, bound, shape)
    # rows behind the last sequence are left as they were
    assert (out[rows:] == 7.0).all()
    # the same call again, on the same workspace: the same bits
    again = cache.attend(s["q"], s["off"], s["ctx"], max(q for q, _ in lens))
    assert torch.equal(again[:rows], got[:rows])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new", [1, 70])
def test_strided_rows_and_pages(types, new):
    """q as columns of a wider buffer, out likewise, pages laid out [page, position, head, 128]."""
    act, kv = TYPES[types]
    s = make([(new, 333), (1, 40), (new, new)], 16, 8, 32, act, kv, seed=3, nhd=True)
    n = s["q"].shape[0]
    wide = torch.randn(n, 32, HD, device="cuda").to(act)
    wide[:, :16] = s["q"]
    dst = torch.zeros(n, 20, HD, dtype=act, device="cuda")
    cache = cache_of(s)
    cache.attend(wide[:, :16], s["off"], s["ctx"], new, scale=0.2, out=dst[:, 4:])
    cache.check()
    want, bound = attend64(s, scale=0.2)
    close(dst[:, 4:], want, bound)
    assert (dst[:, :4] == 0).all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new", [1, 3, 150])
def test_in_place(types, new):
    """The outputs over the queries, items cut between CTAs among them."""
    act, kv = TYPES[types]
    s = make([(new, 3000), (new, 400), (1, 77)], 16, 4, 16, act, kv, seed=14)
    cache = cache_of(s)
    want = cache.attend(s["q"], s["off"], s["ctx"], new)
    q = s["q"].clone()
    got = cache.attend(q, s["off"], s["ctx"], new, out=q)
    cache.check()
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("n", [1, 37, 3000])
@pytest.mark.parametrize("norm", [True, False])
def test_append_matches_64_bits(types, n, norm):
    act, kv = TYPES[types]
    nq, nkv, page, seqs = 16, 8, 16, 5
    per = -(-n // seqs)
    s = make([(0, per + 9)] * seqs, nq, nkv, page, act, kv, seed=n, poison=False)
    g = torch.Generator(device="cuda").manual_seed(n)
    qkv = torch.randn(n, (nq + 2 * nkv) * HD + 8, generator=g, device="cuda").to(act)[:, :-8]   # strided rows
    order = torch.randperm(n, generator=g, device="cuda")
    seq = (order % seqs).to(torch.int32)
    pos = (order // seqs + 9).to(torch.int32)
    if n > 1:
        pos[n // 2] = -1           # a padded row
    ang = torch.arange(per + 9, device="cuda").double()[:, None] * 1e4 ** (-torch.arange(64, device="cuda").double() / 64)
    rope = torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()
    qn = 1 + 0.2 * torch.randn(HD, generator=g, device="cuda") if norm else None
    kn = 1 + 0.2 * torch.randn(HD, generator=g, device="cuda") if norm else None
    k0, v0 = s["k"].clone(), s["v"].clone()
    out = torch.full((n, nq, HD), 3.0, dtype=act, device="cuda")
    cache = cache_of(s)
    cache.append(qkv, seq, pos, rope, qn, kn, eps=1e-6, out=out)
    cache.check()
    (q, qb), (k, kb), v = append64(qkv, seq, pos, rope, qn, kn, 1e-6, nq, nkv)
    live = pos >= 0
    close(out[live], q[live], (qb + q.abs() * HALF[act])[live], "q")
    assert (out[~live] == 3.0).all()
    at = s["table"][seq.long(), pos.long().clamp(min=0) // page].long()
    slot = pos.long().clamp(min=0) % page
    close(s["k"][at, :, slot][live], k[live], (kb + k.abs() * HALF[kv])[live], "k")
    assert torch.equal(s["v"][at, :, slot][live], v.to(kv)[live])
    # nothing else in the pools changed
    rest = torch.ones(k0.shape[0], page, dtype=torch.bool, device="cuda")
    rest[at[live], slot[live]] = False
    for now, was in ((s["k"], k0), (s["v"], v0)):
        assert torch.equal(now.transpose(1, 2)[rest], was.transpose(1, 2)[rest])
    # in place: the queries may go back over the q columns
    again = qkv.clone()
    cache.append(again, seq, pos, rope, qn, kn, eps=1e-6, out=again[:, :nq * HD])
    assert torch.equal(again[:, :nq * HD].reshape(n, nq, HD)[live], out[live])


def _serve(cache, s, qkv, rope, seq, pos, off, ctx, max_q):
    q = cache.append(qkv, seq, pos, rope)
    return cache.attend(q, off, ctx, max_q)


@pytest.mark.parametrize("types", TYPES)
def test_prompt_chunks_then_tokens_equal_one_pass(types):
    """A run as a serving program makes it: prompts in two chunks, then single tokens, every step appended and
    attended, each output against the 64-bit form over what the cache holds; then a draw from logits."""
    import speech_lm_decode_gb300 as q3
    act, kv = TYPES[types]
    nq, nkv, page, lens = 8, 4, 16, [150, 61, 93]
    s = make([(0, 200)] * 3, nq, nkv, page, act, kv, seed=5, poison=False)
    s["k"].fill_(float("nan"))
    s["v"].fill_(float("nan"))
    cache = cache_of(s)
    g = torch.Generator(device="cuda").manual_seed(9)
    ang = torch.arange(200, device="cuda").double()[:, None] * 1e6 ** (-torch.arange(64, device="cuda").double() / 64)
    rope = torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()
    done = [0, 0, 0]
    for counts in ([100, 61, 40], [50, 0, 53], [1, 1, 1], [1, 0, 1], [3, 2, 1]):
        n = sum(counts)
        qkv = torch.randn(n, (nq + 2 * nkv) * HD, generator=g, device="cuda").to(act)
        seq = torch.tensor([i for i, c in enumerate(counts) for _ in range(c)], dtype=torch.int32, device="cuda")
        pos = torch.tensor([done[i] + j for i, c in enumerate(counts) for j in range(c)], dtype=torch.int32,
                           device="cuda")
        done = [d + c for d, c in zip(done, counts)]
        off = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(3)], dtype=torch.int32, device="cuda")
        ctx = torch.tensor(done, dtype=torch.int32, device="cuda")
        q = cache.append(qkv, seq, pos, rope)
        o = cache.attend(q, off, ctx, max(counts))
        cache.check()
        s.update(q=q, off=off, ctx=ctx, lens=list(zip(counts, done)))
        want, bound = attend64(s)
        close(o, want, bound, str(counts))
    assert done == [155, 64, 96] and lens == [150, 61, 93]
    head = torch.randn(nq * HD, 500, generator=g, device="cuda") * 0.05
    logits = o.reshape(o.shape[0], -1).float() @ head
    n = logits.shape[0]
    u = torch.rand(n, generator=g, device="cuda")
    one = torch.ones(n, device="cuda")
    ids, lp = q3.sample_given(logits, u, 0.8 * one, torch.full((n,), 40, dtype=torch.int32, device="cuda"),
                              0.9 * one, 0.05 * one)
    from paged_ref import draw_row
    for i in range(n):
        want, wlp, tol = draw_row(logits[i].cpu().numpy(), float(u[i]), float((0.8 * one)[i]), 40,
                                  float((0.9 * one)[i]), float((0.05 * one)[i]))
        assert int(ids[i]) == want and abs(float(lp[i]) - wlp) <= tol


def test_graph_replay_with_new_lengths():
    """Captured once, replayed with other lengths and values in the same arrays; a second graph of the same
    cache between the replays, and eager calls on another stream."""
    lens = [(1, 400), (1, 17), (1, 1200)]
    s = make([(1, 1200)] * 3, 16, 8, 16, torch.bfloat16, torch.bfloat16, seed=8)
    cache = cache_of(s)
    s["ctx"].copy_(torch.tensor([c for _, c in lens], dtype=torch.int32))
    cache.attend(s["q"], s["off"], s["ctx"], 1)
    torch.cuda.synchronize()
    outs, graphs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(cache.attend(s["q"], s["off"], s["ctx"], 1))
        graphs.append(gr)
    side = torch.cuda.Stream()
    for step in range(4):
        new = [(1, c + 31 * step if c < 1000 else c - 31 * step) for _, c in lens]
        s["ctx"].copy_(torch.tensor([c for _, c in new], dtype=torch.int32))
        s["q"].normal_()
        torch.cuda.synchronize()
        side_out = None
        for gr in graphs:
            gr.replay()
            with torch.cuda.stream(side):
                side_out = cache.attend(s["q"], s["off"], s["ctx"], 1)
        torch.cuda.synchronize()
        cache.check()
        want, bound = attend64({**s, "lens": new})
        for o in outs + [side_out]:
            close(o, want, bound, str(step))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("most", [1, 3, 40])
def test_many_sequences(types, most):
    """More sequences than a CTA has threads, some without new tokens or without any."""
    act, kv = TYPES[types]
    g = torch.Generator().manual_seed(most)
    lens = []
    for _ in range(1500):
        new = int(torch.randint(0, most + 1, (1,), generator=g))
        lens.append((new, int(torch.randint(0, 60, (1,), generator=g))))
    s = make(lens, 2, 1, 16, act, kv, seed=21)
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], most)
    cache.check()
    want, bound = attend64(s)
    close(got, want, bound)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new", [1, 50])
def test_sequences_that_share_pages(types, new):
    act, kv = TYPES[types]
    s = make([(new, 300), (new, 333), (new, 290)], 8, 2, 16, act, kv, seed=22)
    s["table"][1, :12] = s["table"][0, :12]
    s["table"][2, :15] = s["table"][0, :15]
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], new)
    cache.check()
    want, bound = attend64(s)
    close(got, want, bound)


@pytest.mark.parametrize("types", TYPES)
def test_two_streams_at_once(types):
    """Calls of one cache object on two streams, single tokens on one and chunks on the other, beside draws of both
    kinds: the bits of the same calls alone."""
    import speech_lm_decode_gb300 as q3
    act, kv = TYPES[types]
    s = make([(150, 700), (1, 1200), (40, 333)], 16, 8, 16, act, kv, seed=23)
    cache = cache_of(s)
    tokens = torch.randn(3, 16, HD, device="cuda").to(act)
    off1 = torch.arange(4, dtype=torch.int32, device="cuda")
    x = torch.randn(160, 30000, device="cuda")
    f = torch.full((160,), 0.9, device="cuda")
    zero = torch.zeros(160, device="cuda")
    k = torch.zeros(160, dtype=torch.int32, device="cuda")

    def chunks():
        return [cache.attend(s["q"], s["off"], s["ctx"], 150), *q3.sample_given(x, f, f, k, f, zero)]

    def singles():
        return [cache.attend(tokens, off1, s["ctx"], 1), *q3.sample_given(x[:3], f[:3], f[:3], k[:3] + 20, f[:3], zero[:3])]
    want_a, want_b = chunks(), singles()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        with torch.cuda.stream(a):
            got.append((chunks(), want_a))
        with torch.cuda.stream(b):
            got.append((singles(), want_b))
            got.append((singles(), want_b))
    torch.cuda.synchronize()
    cache.check()
    for have, want in got:
        assert all(torch.equal(h, w) for h, w in zip(have, want))


@pytest.mark.parametrize("types", TYPES)
def test_many_row_graph_replay(types):
    """Chunks captured once and replayed with other splits of the rows between the sequences."""
    act, kv = TYPES[types]
    s = make([(90, 700)] * 3, 16, 8, 16, act, kv, seed=12)
    cache = cache_of(s)
    cache.attend(s["q"], s["off"], s["ctx"], 200)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = cache.attend(s["q"], s["off"], s["ctx"], 200)
    for lens in ([(200, 700), (0, 5), (70, 130)], [(1, 1), (128, 128), (141, 699)], [(90, 90), (90, 300), (60, 61)]):
        off = [0, lens[0][0], lens[0][0] + lens[1][0], sum(q for q, _ in lens)]
        s["off"].copy_(torch.tensor(off, dtype=torch.int32))
        s["ctx"].copy_(torch.tensor([c for _, c in lens], dtype=torch.int32))
        s["q"].normal_()
        out.fill_(9.0)
        gr.replay()
        torch.cuda.synchronize()
        cache.check()
        want, bound = attend64({**s, "lens": lens})
        close(out[:off[-1]], want, bound, str(lens))
        assert (out[off[-1]:] == 9.0).all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new", [1, 64])
def test_growing_scores(types, new):
    """Keys whose scores grow along the sequence, by far more than 2^8 from tile to tile: the reference maximum
    moves at every step and the earlier share of the output vanishes."""
    act, kv = TYPES[types]
    s = make([(new, 1500), (new, 640)], 8, 4, 32, act, kv, seed=6)
    direction = torch.randn(HD, device="cuda")
    direction /= direction.norm()
    for i, (_, ctx) in enumerate(s["lens"]):
        pages = s["table"][i, :-(-ctx // 32)].long()
        at = torch.arange(ctx, device="cuda")
        grow = (at.float() / 40.0)[:, None, None] * direction
        k = s["k"][pages[at // 32], :, at % 32].float() * 0.3 + grow
        s["k"][pages[at // 32], :, at % 32] = k.to(kv)
    s["q"].copy_((direction * 12 + 0.3 * torch.randn_like(s["q"].float())).to(act))
    got = cache_of(s).attend(s["q"], s["off"], s["ctx"], new)
    want, bound = attend64(s)
    close(got, want, bound)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("lens", [[(1, 700), (1, 90)], [(3, 700), (2, 90)], [(9, 5000)], [(150, 700), (40, 90)]])
def test_nan_stays_where_it_belongs(lens, types):
    """A query, and a key that a later token sees, that are NaN: NaN in their rows and heads, the rest as ever."""
    act, kv = TYPES[types]
    s = make(lens, 8, 4, 16, act, kv, seed=30)
    cache = cache_of(s)
    n0, ctx = lens[0]
    s["q"][0, 5, 77] = float("nan")
    last = ctx - 1                       # the last token alone sees it
    s["k"][int(s["table"][0, last // 16]), 1, last % 16, 3] = float("nan")
    got = cache.attend(s["q"], s["off"], s["ctx"], n0)
    cache.check()
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[0, 5] = True
    nan[n0 - 1, 2:4] = True
    assert torch.equal(torch.isnan(got), nan)
    clean = dict(s, q=torch.nan_to_num(s["q"]), k=s["k"].clone())
    clean["k"][int(s["table"][0, last // 16]), 1, last % 16, 3] = 0.0
    want, bound = attend64(clean)
    close(torch.where(nan, want.to(act), got), want, bound, "the others")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new", [1, 40])
def test_bad_pages_positions_and_lengths_are_reported(types, new):
    import speech_lm_decode_gb300 as q3
    act, kv = TYPES[types]
    s = make([(new, 100), (new, 90)], 16, 8, 16, act, kv, seed=2, poison=False)
    cache = cache_of(s)
    good = cache.attend(s["q"], s["off"], s["ctx"], new)
    cache.check()
    for bad in (-1, s["k"].shape[0], 2 ** 31 - 1):
        t = s["table"].clone()
        s["table"][0, 2] = bad
        got = cache.attend(s["q"], s["off"], s["ctx"], new)
        with pytest.raises(q3.Q3Error) as e:
            cache.check()
        assert e.value.code == q3.Q3_ERR_BOUNDS
        # the other sequence is not touched by it
        assert torch.equal(got[new:], good[new:])
        s["table"].copy_(t)
    # a context longer than the table, more new tokens than promised, offsets past the rows
    for change in ("ctx", "max_q", "off"):
        ctx, off, mq = s["ctx"].clone(), s["off"].clone(), new
        if change == "ctx":
            ctx[1] = s["table"].shape[1] * 16 + 1
            s["table"].clamp_(max=0)
        elif change == "max_q":
            if new == 1:
                continue
            mq = new - 1
        else:
            off[2] = 2 * new + 3
        cache.attend(s["q"], off, ctx, mq)
        with pytest.raises(q3.Q3Error) as e:
            cache.check()
        assert e.value.code == q3.Q3_ERR_BOUNDS, change
        s["table"].copy_(t)
    # append: a position past the table, a sequence that is none, a page that is none
    qkv = torch.randn(3, 32 * HD, device="cuda").to(act)
    rope = torch.zeros(4096, 64, 2, device="cuda")
    k0 = s["k"].clone()
    s["table"][1, 0] = s["k"].shape[0]
    for seq, pos in (([0, 0, 0], [1 << 20, 4000, 4096]), ([2, -1, 1 << 30], [0, 0, 0]), ([1, 1, 1], [0, 1, 2])):
        cache.append(qkv, torch.tensor(seq, dtype=torch.int32, device="cuda"),
                     torch.tensor(pos, dtype=torch.int32, device="cuda"), rope)
        with pytest.raises(q3.Q3Error) as e:
            cache.check()
        assert e.value.code == q3.Q3_ERR_BOUNDS
    assert torch.equal(s["k"], k0)


def test_pages_past_32_bits():
    """A pool whose offsets pass 2^31 elements: its last pages are written and read."""
    page, nkv = 64, 8
    n_pages = (2 ** 31) // (nkv * page * HD) + 3
    k = torch.empty(n_pages, nkv, page, HD, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    s = make([(1, 100), (70, 101)], 16, nkv, page, torch.bfloat16, torch.bfloat16, seed=4)
    hi = torch.arange(n_pages - s["k"].shape[0], n_pages, device="cuda")
    k[hi], v[hi] = s["k"], s["v"]
    ok = s["table"] < s["k"].shape[0]
    s["table"][ok] += int(hi[0])
    s.update(k=k, v=v)
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], 70)
    one = cache.attend(s["q"][:1], torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda"), s["ctx"], 1)
    cache.check()
    want, bound = attend64(s)
    close(got, want, bound)
    close(one, want[:1], bound[:1])
    qkv = torch.randn(2, 32 * HD, device="cuda").to(torch.bfloat16)
    rope = torch.zeros(200, 64, 2, device="cuda")
    rope[..., 0] = 1
    cache.append(qkv, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                 torch.tensor([99, 100], dtype=torch.int32, device="cuda"), rope)
    cache.check()
    for i, p in ((0, 99), (1, 100)):
        at = int(s["table"][i, p // page])
        assert torch.equal(v[at, :, p % page], qkv.view(2, 32, HD)[i, 24:])
        assert torch.equal(k[at, :, p % page], qkv.view(2, 32, HD)[i, 16:24])


def test_refusals():
    import speech_lm_decode_gb300 as q3
    s = make([(1, 30)], 16, 8, 16, torch.bfloat16, torch.bfloat16, seed=1)
    cache = cache_of(s)
    with pytest.raises(ValueError):
        q3.PagedKV(s["k"], s["v"].float(), s["table"], 16)
    with pytest.raises(ValueError):
        q3.PagedKV(s["k"], s["v"], s["table"].long(), 16)
    with pytest.raises(ValueError):
        q3.PagedKV(s["k"].half(), s["v"].half(), s["table"], 16)
    with pytest.raises(q3.Q3Error):
        q3.PagedKV(s["k"], s["v"], s["table"], 12)
    with pytest.raises(ValueError):
        cache.attend(s["q"].half(), s["off"], s["ctx"], 1)
    with pytest.raises(ValueError):
        cache.attend(s["q"], s["off"].long(), s["ctx"], 1)
    with pytest.raises(ValueError):
        cache.attend(s["q"][..., :64], s["off"], s["ctx"], 1)
    with pytest.raises(q3.Q3Error):
        cache.attend(s["q"], s["off"], s["ctx"], 1, scale=0.0)
    with pytest.raises(q3.Q3Error):
        cache.attend(s["q"], s["off"], s["ctx"], -1)
    wide = torch.zeros(3, 16 * HD + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(q3.Q3Error):     # rows that do not start on 16-byte boundaries
        cache.attend(wide[:, 4:], s["off"], s["ctx"], 1)
    f32 = q3.PagedKV(s["k"].float(), s["v"].float(), s["table"], 16)
    with pytest.raises(q3.Q3Error):     # bf16 activations over fp32 pages
        f32.attend(s["q"], s["off"], s["ctx"], 1)
    # broadcast tensors: their rows, pages or heads are the same memory
    with pytest.raises(ValueError):
        cache.attend(s["q"][:1].expand(5, 16, HD), s["off"], s["ctx"], 1)
    with pytest.raises(ValueError):
        cache.attend(s["q"], s["off"], s["ctx"], 1, out=torch.empty_like(s["q"][:1]).expand(len(s["q"]) + 1, 16, HD))
    with pytest.raises(ValueError):
        q3.PagedKV(s["k"][:1].expand(9, 8, 16, HD), s["v"][:1].expand(9, 8, 16, HD), s["table"], 16)
    with pytest.raises(ValueError):
        q3.PagedKV(s["k"][:, :1].expand(-1, 8, 16, HD), s["v"][:, :1].expand(-1, 8, 16, HD), s["table"], 16)
    # nothing to do is no error
    assert cache.attend(s["q"][:0], torch.zeros(2, dtype=torch.int32, device="cuda"), s["ctx"], 1).shape == (0, 16, HD)
