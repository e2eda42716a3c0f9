"""Paged attention where a call goes wrong or to an extreme: offsets, pages, scales, waits that run out; and what cache
objects share."""
import pytest

torch = pytest.importorskip("torch")

from paged_ref import HD, attend64, make  # noqa: E402
from test_gpu_paged import TYPES, cache_of, close  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new", [1, 3, 40])
def test_offsets_whose_difference_wraps_around(new, types):
    """Offsets of any value: 2^31 - 1 to -2^31 is one row further in 32 bits, and no row of the call."""
    import speech_lm_decode_gb300 as q3
    act, kv = TYPES[types]
    s = make([(new, 100), (0, 50), (0, 60), (0, 70), (0, 80)], 8, 4, 16, act, kv, seed=40, extra_rows=3)
    want, bound = attend64({**s, "lens": [(new, 100)]})
    cache = cache_of(s)
    top, low = 2 ** 31 - 1, -2 ** 31
    for off in ([0, new, top, low, low + 1, 0], [0, new, low, top, low, top], [0, new, new + 4, new - 1, top - 1, low],
                [0, new, top, low, top, low]):
        out = torch.full_like(s["q"], 7.0)
        cache.attend(s["q"], torch.tensor(off, dtype=torch.int32, device="cuda"), s["ctx"], new, out=out)
        with pytest.raises(q3.Q3Error) as e:
            cache.check()
        assert e.value.code == q3.Q3_ERR_BOUNDS
        close(out[:new], want, bound, str(off))
        assert (out[new:] == 7.0).all(), off


def attend_seen(s, gone, scale=HD ** -0.5):
    """attend64 with keys that do not count: gone[i] has the page indices of sequence i that are out of range."""
    out, bound = [], []
    for i, (n_new, ctx) in enumerate(s["lens"]):
        there = torch.tensor([j for j in range(ctx) if j // s["page"] not in gone[i]], dtype=torch.long, device="cuda")
        pages = s["table"][i, :-(-ctx // s["page"])].long()
        pages = torch.where(pages.clamp(0, s["k"].shape[0] - 1) == pages, pages, 0)
        k, v = (p[pages].transpose(1, 2).reshape(-1, s["nkv"], HD)[there].double() for p in (s["k"], s["v"]))
        q = s["q"][int(s["off"][i]):int(s["off"][i]) + n_new].double()
        last = ctx - n_new + torch.arange(n_new, device="cuda")
        hidden = there[None] > last[:, None]
        some = ~hidden.all(1)
        o = torch.zeros(n_new, s["nq"], HD, dtype=torch.float64, device="cuda")
        b = torch.zeros_like(o)
        for h in range(s["nq"] if len(there) else 0):
            kh, vh = k[:, h * s["nkv"] // s["nq"]], v[:, h * s["nkv"] // s["nq"]]
            p = torch.softmax((q[:, h] @ kh.T * scale).masked_fill(hidden, float("-inf")), -1)
            p[~some] = 0
            o[:, h] = p @ vh
            # as in attend64: the operands' and the sums' errors of a score, twice; parts, exp and sums of the weights
            e_s = scale * (q[:, h].abs() @ kh.abs().T).masked_fill(hidden, 0).amax(-1) * 2.0 ** -16
            e_p = 2.0 ** -17 + 2.0 ** -20 + (ctx + 128) * 2.0 ** -24 + (2.0 ** -8 if s["q"].dtype != torch.float32 else 0)
            b[:, h] = (p @ vh.abs()) * (2 * e_s + e_p)[:, None]
        out.append(o)
        bound.append(b + o.abs() * (2.0 ** -24 if s["q"].dtype == torch.float32 else 2.0 ** -8))
    return torch.cat(out), torch.cat(bound)


# (new tokens, positions) of each sequence and the pages of each that are out of range
GONE = {
    "single": ([(1, 300), (1, 90)], [{2, 18}, {0}]),
    "few": ([(3, 700), (2, 40)], [{0, 1, 2, 43}, {1}]),
    "chunk": ([(40, 700), (17, 333)], [{2, 3, 11, 43}, set(range(8, 16))]),
    "two-tiles": ([(150, 700), (200, 1100)], [{0, 20}, {5, 6, 7, 40, 68}]),
    "all-of-one": ([(9, 150), (30, 400)], [set(range(10)), {24}]),
    "long": ([(20, 9000), (1, 64)], [{0, 7, 100, 562}, {3}]),
}


def check_gone(case, types, page):
    """Whichever kernel serves the call: such a page's keys are masked, rows that see nothing else are zeros, and no
    other page is read in its place (page 0 belongs to nobody and holds NaN)."""
    import speech_lm_decode_gb300 as q3
    act, kv = TYPES[types]
    lens, gone = GONE[case]
    if page == 128:
        gone = [{j * 16 // page for j in g} for g in gone]
    s = make(lens, 8, 4, page, act, kv, seed=41)
    # what page 0 holds moves to a page that no sequence has
    to = next(i for i in range(s["k"].shape[0]) if not (s["table"] == i).any())
    if to != 0:
        s["k"][to], s["v"][to] = s["k"][0].clone(), s["v"][0].clone()
        s["table"][s["table"] == 0] = to
        s["k"][0], s["v"][0] = float("nan"), float("nan")
    bad = [-1, s["k"].shape[0], 2 ** 31 - 1, -2 ** 31]
    for i, g in enumerate(gone):
        for n, j in enumerate(sorted(g)):
            s["table"][i, j] = bad[n % 4]
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], max(q for q, _ in lens))
    with pytest.raises(q3.Q3Error) as e:
        cache.check()
    assert e.value.code == q3.Q3_ERR_BOUNDS
    want, bound = attend_seen(s, gone)
    close(got, want, bound, case)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("types", ["bf16", "f32"])
@pytest.mark.parametrize("case", GONE)
def test_keys_of_pages_out_of_range_do_not_count(case, types, page):
    check_gone(case, types, page)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("case", GONE)
def test_keys_of_fp32_pages_out_of_range_do_not_count(case, page):
    check_gone(case, "f32kv", page)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new", [1, 3, 40, 150])
@pytest.mark.parametrize("scale", [1e-38, 1.4e-45, 1e-30])
def test_scales_next_to_zero(scale, new, types):
    """Every score is the same then: the outputs are means of the values."""
    act, kv = TYPES[types]
    s = make([(new, 700), (new, 40), (1, 300)], 8, 4, 16, act, kv, seed=42)
    cache = cache_of(s)
    got = cache.attend(s["q"], s["off"], s["ctx"], new, scale=scale)
    cache.check()
    want, bound = attend64(s, scale=scale)
    close(got, want, bound, str(scale))


def test_cache_objects_share_the_workspace_of_a_stream():
    """28 layers' caches on a stream hold one workspace, another stream's calls another; calls of unlike caches in
    turn give the bits of each alone; what the last object held is given back."""
    import gc
    import speech_lm_decode_gb300 as q3
    states = [make([(new, 900), (new, 70)], 8, nkv, 16, *TYPES[t], seed=43) for t in TYPES for new, nkv in ((1, 8), (40, 2))]
    news = [1, 40] * 3
    alone = []
    for s, new in zip(states, news):
        alone.append(cache_of(s).attend(s["q"], s["off"], s["ctx"], new))
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    caches = [cache_of(s) for s in states * 5]
    got = [c.attend(s["q"], s["off"], s["ctx"], new) for _ in range(2) for c, s, new in zip(caches, states * 5, news * 5)]
    one = caches[0].ws_bytes
    assert torch.cuda.memory_allocated() - before < 1.5 * one
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got += [c.attend(s["q"], s["off"], s["ctx"], new) for c, s, new in zip(caches, states, news)]
    assert one < torch.cuda.memory_allocated() - before < 2.5 * one
    torch.cuda.synchronize()
    for c in caches:
        c.check()
    for i, o in enumerate(got):
        assert torch.equal(o, alone[i % len(alone)])
    del c, caches, got, o
    gc.collect()
    assert torch.cuda.memory_allocated() - before < one / 2


@pytest.mark.parametrize("types", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(150, 3000), (40, 333)], [(40, 900), (17, 64), (1, 500)]])
def test_a_wait_that_runs_out(lens, types):
    """Every CTA's wait for room for its n-th tile counts as run out, at the start of an item or inside: the call returns,
    says so, and leaves counters with which the next call on the workspace gives the bits that it should."""
    import speech_lm_decode_gb300 as q3
    act, kv = TYPES[types]
    s = make(lens, 8, 4, 16, act, kv, seed=44)
    most = max(q for q, _ in lens)
    cache = cache_of(s)
    want = cache.attend(s["q"], s["off"], s["ctx"], most)
    cache.check()
    (ws,) = cache._ws.values()
    for n in list(range(1, 14)) + [20, 33]:
        broken = q3.PagedKV(s["k"], s["v"], s["table"], n_q_heads=8, inject_timeout=n)
        broken.attend(s["q"], s["off"], s["ctx"], most)
        torch.cuda.synchronize()
        e = int(broken.err.item())
        assert e in (0, q3.Q3PAGED_ERR_TIMEOUT) and (e or n > 2)     # (a CTA may have fewer tiles than that)
        assert list(broken._ws.values())[0] is ws
        assert not ws[:q3.Q3PAGED_COUNTER_BYTES].any()
        assert torch.equal(cache.attend(s["q"], s["off"], s["ctx"], most), want)
        cache.check()
    with pytest.raises(q3.Q3Error):
        q3.PagedKV(s["k"], s["v"], s["table"], n_q_heads=8, inject_timeout=-1)
