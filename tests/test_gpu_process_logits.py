"""Penalties, biases and masks on logits against their definition in 64 bits, alone and in front of the draw."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged8_ref import HALF, process64  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def case(n, vocab, dtype, seed, history=0, biases=0, masks=0, rows=False):
    """Keyword arguments on the GPU (and logits) of a call; ids repeat, also among the biases."""
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.standard_normal((n, vocab)).astype(np.float32) * 3).to(dtype).cuda()
    kw = {}

    def dev(a, t=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    if history:
        h = (g.random((n, history)) ** 2 * vocab).astype(np.int32)
        h[:, ::7] = -1
        if vocab > 3:
            h[:, 1::5] = vocab - 1
        kw["history"] = dev(h)
        nh = g.integers(0, history + 1, n)
        nh[0] = history
        kw["n_history"] = dev(nh)
        kw["n_prompt"] = dev(g.integers(0, history + 1, n))
        kw["repetition"] = dev(0.5 + g.random(n), torch.float32)
        kw["presence"] = dev(g.standard_normal(n), torch.float32)
        kw["frequency"] = dev(g.standard_normal(n) * 0.3, torch.float32)
    if biases:
        count = g.integers(0, biases + 1, n)
        count[-1] = biases
        off = np.concatenate(([0], np.cumsum(count)))
        kw["bias_off"], kw["bias_ids"] = dev(off), dev((g.random(off[-1]) ** 2 * vocab).astype(np.int32))
        kw["bias"] = dev(g.standard_normal(off[-1]) * 2, torch.float32)
    if masks:
        w = g.integers(-2 ** 31, 2 ** 31, (masks, (vocab + 31) // 32), dtype=np.int64).astype(np.int32)
        w[0] = 0
        w[-1] = -1
        kw["mask"] = dev(w)
        if rows or masks < n:
            kw["mask_row"] = dev(g.integers(-1, masks, n))
    return x, kw


def check(x, kw, got):
    host = {k: v.cpu().numpy() for k, v in kw.items()}
    want, bound = process64(x.float().cpu().numpy(), **host)
    y = got.float().cpu().double().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(y[~fine], want[~fine])
    err = np.abs(y[fine] - want[fine])
    lim = bound[fine] + (np.abs(want[fine]) + bound[fine]) * HALF[x.dtype] + 1e-40
    assert (err <= lim).all(), float((err / lim).max())
    # what no history, bias or mask names is the logit's own bits
    same = want == x.float().cpu().double().numpy()
    assert np.array_equal(y[same], want[same])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 33, 1000, 2048, 8191, 8193, 50257, 151936, 262144])
@pytest.mark.parametrize("what", ["history", "biases", "masks", "all"])
def test_matches_64_bits(what, vocab, dtype):
    import speech_lm_decode_gb300 as q3
    n = 7 if vocab < 50000 else 3
    x, kw = case(n, vocab, TYPES[dtype], vocab, **{"history": dict(history=500), "biases": dict(biases=40),
                 "masks": dict(masks=n), "all": dict(history=900, biases=30, masks=3, rows=True)}[what])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    was = x.clone()
    got = q3.process_logits(x, **kw, err=err)
    assert torch.equal(x, was) and int(err) == 0
    check(x, kw, got)
    # in place, on strided rows: the same bits
    wide = torch.zeros(n, vocab + 24, dtype=TYPES[dtype], device="cuda")
    wide[:, 8:8 + vocab] = x
    inner = wide[:, 8:8 + vocab]
    assert q3.process_logits(inner, **kw, out=inner, err=err) is inner
    assert torch.equal(inner, got) and not wide[:, :8].any() and not wide[:, 8 + vocab:].any()
    # rows at odd places, and outputs that lie otherwise in memory than the logits
    odd = torch.zeros(n, vocab + 3, dtype=TYPES[dtype], device="cuda")
    odd[:, 1:1 + vocab] = x
    assert torch.equal(q3.process_logits(odd[:, 1:1 + vocab], **kw, err=err), got)
    into = torch.zeros(n, vocab + 5, dtype=TYPES[dtype], device="cuda")
    q3.process_logits(x, **kw, out=into[:, 3:3 + vocab], err=err)
    assert torch.equal(into[:, 3:3 + vocab], got) and not into[:, :3].any() and not into[:, 3 + vocab:].any()
    # in place at odd places
    assert torch.equal(q3.process_logits(odd[:, 1:1 + vocab], **kw, out=odd[:, 1:1 + vocab]), got)
    assert not odd[:, :1].any() and not odd[:, 1 + vocab:].any()
    assert int(err) == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_parts_that_are_left_out(dtype):
    import speech_lm_decode_gb300 as q3
    x, kw = case(5, 3001, TYPES[dtype], 3, history=80, biases=20, masks=5)
    assert torch.equal(q3.process_logits(x), x)
    assert q3.process_logits(x, out=x) is x
    for names in (("history", "n_history", "repetition"), ("history", "n_history", "n_prompt", "presence"),
                  ("history", "n_history", "frequency"), ("history", "n_history", "n_prompt"), ("bias_off", "bias_ids", "bias"),
                  ("mask",), ("history", "n_history", "n_prompt", "repetition", "mask")):
        part = {k: kw[k] for k in names}
        check(x, part, q3.process_logits(x, **part))
    # none of a thing: an empty history, no biases
    none = {**{k: kw[k] for k in ("n_history", "repetition")}, "history": kw["history"][:, :0],
            "bias_off": torch.zeros(6, dtype=torch.int32, device="cuda"), "bias_ids": kw["bias_ids"][:0], "bias": kw["bias"][:0]}
    assert torch.equal(q3.process_logits(x, **none), x)


@pytest.mark.parametrize("dtype", TYPES)
def test_long_histories(dtype):
    """Histories that are longer than a slice of the vocabulary; one id said thousands of times."""
    import speech_lm_decode_gb300 as q3
    x, kw = case(3, 20000, TYPES[dtype], 5, history=40000, biases=3000)
    kw["history"][1, :] = 19999
    kw["frequency"].fill_(0.001)
    check(x, kw, q3.process_logits(x, **kw))


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan(dtype):
    import speech_lm_decode_gb300 as q3
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[inf, -inf, nan, 1.0, -0.0, inf, nan, 2.0]], dtype=TYPES[dtype], device="cuda")
    h = torch.tensor([[0, 1, 2, 3, 4, 3]], dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    kw = dict(history=h, n_history=one.int() * 6, repetition=one * 2.0, presence=one * 0.5, frequency=one * 0.25,
              bias_off=torch.tensor([0, 4], dtype=torch.int32, device="cuda"),
              bias_ids=torch.tensor([1, 3, 7, 7], dtype=torch.int32, device="cuda"),
              bias=torch.tensor([5.0, inf, 1.0, 1.0], device="cuda"),
              mask=torch.tensor([[0b10011111]], dtype=torch.int32, device="cuda"))
    got = q3.process_logits(x, **kw).float().cpu()[0]
    assert got[0] == inf and got[1] == -inf and torch.isnan(got[2]) and got[3] == inf and got[4] == -0.75
    assert got[5] == -inf and got[6] == -inf and got[7] == 4.0


def test_the_biases_of_an_id_are_added_in_their_order():
    import speech_lm_decode_gb300 as q3
    x = torch.zeros(1, 100, device="cuda")
    vals = [1e8, 1.0, -1e8, 3.0, 1e-3] * 7
    ids = [42] * len(vals)
    want = np.float32(0)
    for v in vals:
        want = np.float32(want + np.float32(v))
    kw = dict(bias_off=torch.tensor([0, len(vals)], dtype=torch.int32, device="cuda"),
              bias_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"), bias=torch.tensor(vals, device="cuda"))
    for _ in range(5):
        got = q3.process_logits(x, **kw)
        assert float(got[0, 42]) == float(want) and got.count_nonzero() <= 1


def test_what_is_out_of_range_is_reported_and_skipped():
    import speech_lm_decode_gb300 as q3
    x, kw = case(4, 500, torch.float32, 8, history=50, biases=10, masks=2, rows=True)
    for name, at, bad in (("history", (0, 3), 500), ("history", (0, 3), 2 ** 31 - 1), ("n_history", 1, 51), ("n_history", 1, -1),
                          ("bias_ids", -1, 500), ("bias_ids", -1, -1), ("bias_ids", -1, -2 ** 31), ("bias_off", 2, 10 ** 6),
                          ("bias_off", 2, -1), ("bias_off", 4, 2 ** 31 - 1), ("mask_row", 2, 2), ("mask_row", 2, -2)):
        part = {k: v.clone() for k, v in kw.items()}
        part["n_history"][0] = 50
        part[name][at] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = q3.process_logits(x, **part, err=err)
        assert int(err) == q3.Q3PAGED_ERR_BOUNDS, (name, bad)
        check(x, part, got)
        q3.process_logits(x, **part)          # without an error word
        if name == "mask_row":
            assert (got[2] == float("-inf")).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_in_front_of_the_draw_in_a_graph(dtype):
    """A masked, penalised batch drawn from, eager and replayed with new histories; a row without allowed ids draws -1."""
    import speech_lm_decode_gb300 as q3
    n, vocab = 6, 9000
    x, kw = case(n, vocab, TYPES[dtype], 9, history=64, biases=12, masks=4, rows=True)
    kw["mask_row"].copy_(torch.tensor([0, 1, 2, 3, -1, 1], dtype=torch.int32))     # mask 0 allows nothing
    f = dict(temperature=torch.ones(n, device="cuda"), top_k=torch.full((n,), 40, dtype=torch.int32, device="cuda"),
             top_p=torch.full((n,), 0.9, device="cuda"), min_p=torch.zeros(n, device="cuda"))
    u = torch.rand(n, device="cuda")

    def step():
        return q3.sample_given(q3.process_logits(x, **kw), u, **f)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        kw["n_history"].copy_(torch.randint(0, 65, (n,), dtype=torch.int32))
        u.copy_(torch.rand(n))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1].nan_to_num(7.0), want[1].nan_to_num(7.0))
        ids = got[0].cpu().numpy()
        assert ids[0] == -1
        for r in range(1, n):
            m = int(kw["mask_row"][r])
            assert m < 0 or int(kw["mask"][m, ids[r] // 32]) >> int(ids[r] % 32) & 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [40, 700])
def test_many_rows(rows, dtype):
    """Batches whose parts do not all run at once: copying and the named ids in kernels of their own; histories that
    their table does not take, empty ones, and rows without a mask beside those with one."""
    import speech_lm_decode_gb300 as q3
    x, kw = case(rows, 60000 if rows == 40 else 9001, TYPES[dtype], rows, history=300, biases=20, masks=5, rows=True)
    got = q3.process_logits(x, **kw)
    check(x, kw, got)
    y = x.clone()
    assert torch.equal(q3.process_logits(y, **kw, out=y), got)
    part = {k: v for k, v in kw.items() if not k.startswith("mask")}
    check(x, part, q3.process_logits(x, **part))
    y = x.clone()
    check(x, part, q3.process_logits(y, **part, out=y))
    part = {k: v for k, v in kw.items() if k.startswith("bias") or k.startswith("mask")}
    check(x, part, q3.process_logits(x, **part))


def test_more_biases_than_the_table_takes():
    import speech_lm_decode_gb300 as q3
    x, kw = case(40, 60000, torch.float32, 12, history=300, biases=9000)
    kw["bias_off"] = torch.tensor([0, 9000] + [9000] * 38 + [int(kw["bias_off"][-1])], dtype=torch.int32, device="cuda")
    kw["bias_ids"], kw["bias"] = kw["bias_ids"][:int(kw["bias_off"][-1])], kw["bias"][:int(kw["bias_off"][-1])]
    kw["bias_off"][-1] = 9300
    check(x, kw, q3.process_logits(x, **kw))


def test_two_streams_at_once_and_what_follows():
    """Calls on two streams with the draw behind each: it sees the whole of its logits."""
    import speech_lm_decode_gb300 as q3
    sets = [case(60, 50000, torch.bfloat16, seed, history=200, biases=9, masks=60) for seed in (13, 14)]
    n = 60
    f = (torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"), torch.ones(n, device="cuda"), torch.zeros(n, device="cuda"))
    u = torch.rand(n, device="cuda")
    want = [q3.process_logits(x, **kw) for x, kw in sets]
    ids = [q3.sample_given(w, u, *f)[0] for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(15):
        for i, (x, kw) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                y = q3.process_logits(x, **kw)
                got[i].append((q3.sample_given(y, u, *f)[0], y.float().nan_to_num(0, 0, -1e4).sum(1), y))
    torch.cuda.synchronize()
    # the same in a graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = q3.process_logits(sets[0][0], **sets[0][1])
        drawn = q3.sample_given(y, u, *f)[0]
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(drawn, ids[0])
    for i in range(2):
        s = want[i].float().nan_to_num(0, 0, -1e4).sum(1)
        assert all(torch.equal(a, ids[i]) and torch.equal(b, s) and torch.equal(c, want[i]) for a, b, c in got[i])


def test_refusals():
    import speech_lm_decode_gb300 as q3
    x, kw = case(4, 500, torch.float32, 10, history=50, biases=10, masks=4)
    for bad in (dict(logits=x.cpu()), dict(logits=x.half()), dict(logits=x.t()), dict(logits=x[0]), dict(history=kw["history"].long()),
                dict(history=kw["history"][:3]), dict(n_history=kw["n_history"][:3]), dict(repetition=kw["repetition"].double()),
                dict(bias=kw["bias"][:-1]), dict(bias_off=kw["bias_off"][:-1]), dict(mask=kw["mask"][:, :-1]),
                dict(mask=kw["mask"].long()), dict(out=x.bfloat16()), dict(out=x[:, :-1]), dict(out=x[:1].expand(4, 500)),
                dict(err=torch.zeros(1, device="cuda"))):
        a = {**kw, **bad}
        logits = a.pop("logits", x)
        with pytest.raises(ValueError):
            q3.process_logits(logits, **a)
    for drop in (("history",), ("bias",), ("bias_off",), ("bias_ids", "bias"), ("n_history",)):
        with pytest.raises(q3.Q3Error):
            q3.process_logits(x, **{k: v for k, v in kw.items() if k not in drop})
    with pytest.raises(q3.Q3Error):
        q3.process_logits(x, mask=kw["mask"][:3])                       # three masks for four rows
    with pytest.raises(q3.Q3Error):
        q3.process_logits(x, mask_row=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert q3.process_logits(x[:0]).shape == (0, 500)
