"""The draw from given uniform numbers against its definition: ids have to be equal, on every row."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_ref import draw_row  # noqa: E402

pytestmark = pytest.mark.gpu


def run(x, u, t, k, p, mp):
    import speech_lm_decode_gb300 as q3
    n = x.shape[0]

    def dev(a, dt):
        return torch.as_tensor(np.broadcast_to(np.asarray(a), (n,)).copy()).to(dt).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, lp = q3.sample_given(x, dev(u, torch.float32), dev(t, torch.float32), dev(k, torch.int32),
                              dev(p, torch.float32), dev(mp, torch.float32), err=err)
    return ids.cpu().numpy(), lp.cpu().numpy(), int(err.item())


def check(x, u, t, k, p, mp):
    ids, lp, err = run(x, u, t, k, p, mp)
    n = x.shape[0]
    xs = x.float().cpu().numpy()
    u, t, k, p, mp = (np.broadcast_to(np.asarray(a), (n,)) for a in (u, t, k, p, mp))
    bad = False
    for i in range(n):
        want, wlp, tol = draw_row(xs[i], np.float32(u[i]), np.float32(t[i]), int(k[i]), np.float32(p[i]),
                                  np.float32(mp[i]))
        assert ids[i] == want, (i, ids[i], want)
        if want < 0:
            bad = True
            assert np.isnan(lp[i])
        else:
            assert abs(lp[i] - wlp) <= tol, (i, lp[i], wlp)
    assert err == (1 if bad else 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 33, 1000, 2048, 4097, 20000, 151936])
def test_filters(vocab, dtype):
    g = torch.Generator().manual_seed(vocab)
    n = 24 if vocab < 50000 else 12
    x = (torch.randn(n, vocab, generator=g) * 3).to(dtype)
    if vocab > 40:
        x[:, torch.randint(0, vocab, (vocab // 20,), generator=g)] = float("-inf")
        x[:, vocab // 3] = 0.5
    rng = np.random.default_rng(vocab)
    k = rng.choice([0, 1, 2, 50, 400, vocab, vocab + 5], n)
    p = rng.choice([1.0, 0.95, 0.5, 0.1, 0.999], n)
    mp = rng.choice([0.0, 0.0, 0.05, 0.5, 1.0], n)
    t = rng.choice([1.0, 0.7, 1.3, 0.0, 0.05, 8.0], n)
    check(x.cuda(), rng.random(n).astype(np.float32), t, k, p, mp)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_largest_vocabulary_and_many_rows(dtype):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(5, 262144, generator=g) * 2).to(dtype)
    u = np.linspace(0.02, 0.98, 5, dtype=np.float32)
    for k, p in ((0, 0.9), (60, 1.0), (300, 0.8)):
        check(x.cuda(), u, 0.8, k, p, 0.001)
    # more rows than the GPU holds at once
    x = (torch.randn(700, 9001, generator=g) * 2).to(dtype)
    check(x.cuda(), (np.arange(700) / 700).astype(np.float32), 1.0, np.arange(700) % 200, 0.9, 0.0)


# (rows, vocabulary) past what shared memory holds while all rows run at once: one, two and four CTAs a row
STREAMED = [(160, 33000), (80, 50001), (40, 90000)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab", STREAMED)
def test_many_rows_of_large_vocabularies(n, vocab, dtype):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, vocab, generator=g) * torch.linspace(0.1, 5, n)[:, None]
    x[:, torch.randint(0, vocab, (vocab // 20,), generator=g)] = float("-inf")
    rng = np.random.default_rng(vocab)
    k = rng.choice([0, 0, 1, 50, 400, 5000, vocab, vocab + 5], n)
    p = rng.choice([1.0, 0.95, 0.95, 0.5, 0.999, 0.0], n)
    mp = rng.choice([0.0, 0.0, 0.05, 0.5, 1.0], n)
    t = rng.choice([1.0, 0.7, 1.3, 0.0, 0.05, 8.0], n)
    check(x.to(dtype).cuda(), rng.random(n).astype(np.float32), t, k, p, mp)


@pytest.mark.parametrize("n,vocab", STREAMED)
def test_many_rows_of_awkward_logits(n, vocab):
    """What the tests below do to a few rows: ties, crowded borders, extreme quotients, rows that fail, and rows that
    do not start on 16-byte boundaries."""
    g = torch.Generator().manual_seed(n + 1)
    wide = torch.randint(-3, 4, (n, vocab + 7), generator=g).float() * 0.5
    x = wide[:, 3:3 + vocab]
    t = np.ones(n, np.float32)
    x[0::10] = torch.randn(len(x[0::10]), vocab, generator=g) * 0.01
    x[1::10] = 1.25
    x[2::10] = torch.linspace(-90, 0, vocab)
    x[3::10] = torch.linspace(0, 1e-3, vocab)
    x[4::10] = torch.randn(len(x[4::10]), vocab, generator=g) * 1e25
    t[4::10] = 1e-5
    x[5::10] = torch.randn(len(x[5::10]), vocab, generator=g) * 1e-30
    t[5::10] = 1e10
    x[6::10] = torch.where(torch.arange(vocab) % 2 == 0, 0.0, -0.0)
    x[7, 17], x[17, vocab - 1], x[27] = float("nan"), float("inf"), float("-inf")
    x[8::10, vocab // 2] = 9.0
    t[9], t[19], t[29] = -1, np.inf, np.nan
    u = np.linspace(0, 1, n, dtype=np.float32)
    u[-1] = np.float32(1 - 2.0 ** -24)
    rng = np.random.default_rng(n)
    k = rng.choice([0, 0, 0, 7, 150, 900], n)
    p = rng.choice([1.0, 0.9, 0.6, 0.3, 0.999], n)
    mp = rng.choice([0.0, 0.0, 0.4], n)
    check(wide.cuda()[:, 3:3 + vocab], u, t, k, p, mp)


@pytest.mark.parametrize("vocab", [300, 5000, 70000])
def test_ties_and_edges(vocab):
    """Few distinct values (ties at every threshold, ids of the same value kept from the lowest on), uniform
    logits, +-0, u at both ends."""
    g = torch.Generator().manual_seed(vocab + 1)
    x = torch.randint(-3, 4, (20, vocab), generator=g).float() * 0.5
    x[3] = 1.25
    x[4] = torch.where(torch.arange(vocab) % 2 == 0, 0.0, -0.0)
    x[5] = -1e30
    x[5, vocab // 2] = 3e30
    x[6] = float("-inf")
    x[6, vocab - 1] = -5.0
    x[7] = torch.linspace(-90, 0, vocab)
    u = np.linspace(0, 1, 20, dtype=np.float32)
    u[-1] = np.float32(1 - 2.0 ** -24)
    for k, p, mp in ((0, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.6, 0.0), (150, 0.3, 0.0), (0, 1.0, 0.4), (0, 0.0, 0.0),
                     (0, -1.0, 0.0), (0, 0.9, 2.0), (0, float("nan"), 0.0), (0, 0.7, float("nan")), (3, 0.99, 1.0)):
        check(x.cuda(), u, 1.0, k, p, mp)


def test_rows_that_fail():
    x = torch.randn(9, 3000, generator=torch.Generator().manual_seed(2))
    x[0, 17] = float("nan")
    x[1, 2999] = float("inf")
    x[2] = float("-inf")
    x[5, 0] = 3e38
    t = np.array([1, 1, 1, -1, np.nan, 0.5, 0, 1, 1e-3], np.float32)   # 5: the quotient overflows
    check(x.cuda(), 0.3, t, 40, 0.9, 0.0)


def test_extreme_temperatures_and_logits():
    """Quotients that are denormal (many logits share one), that underflow to zero, an infinite temperature (uniform,
    or no number where a logit is -inf), and logits that the quick division does not take."""
    g = torch.Generator().manual_seed(8)
    x = torch.randn(10, 5000, generator=g)
    x[1] *= 1e-30
    x[2] *= 1e-38
    x[3] *= 1e25
    x[4] = torch.where(torch.rand(5000, generator=g) < 0.5, x[4] * 1e-25, x[4] * 1e20)
    x[6, 3000] = float("-inf")
    x[8] *= 2.0 ** 70
    t = np.array([1e12, 1e10, 1.0, 1e-5, 3.0, np.inf, np.inf, 3e38, 2.0 ** 60, 2.0 ** -40], np.float32)
    u = np.linspace(0.05, 0.95, 10, dtype=np.float32)
    for k, p in ((0, 1.0), (40, 1.0), (200, 0.9), (0, 0.7)):
        check(x.cuda(), u, t, k, p, 0.0)


@pytest.mark.parametrize("vocab", [3000, 40000])
def test_many_ids_at_the_border(vocab):
    """Crowded borders: hundreds of equal or nearly equal logits where top-k or top-p cuts, beyond what the lists
    hold."""
    g = torch.Generator().manual_seed(vocab)
    x = torch.randn(6, vocab, generator=g) * 0.01
    x[1] = torch.randint(0, 3, (vocab,), generator=g).float()
    x[2] = 2.0
    x[3, : vocab // 2] = 1.0
    x[4] = torch.linspace(0, 1e-3, vocab)
    u = np.linspace(0.01, 0.99, 6, dtype=np.float32)
    for k, p in ((100, 1.0), (700, 1.0), (0, 0.5), (900, 0.33), (0, 0.999)):
        check(x.cuda(), u, 1.0, k, p, 0.0)


def test_strided_rows_and_graph():
    import speech_lm_decode_gb300 as q3
    wide = torch.randn(16, 5007, device="cuda")
    x = wide[:, 3:4803]
    check(x, np.linspace(0, 0.99, 16, dtype=np.float32), 0.9, 50, 0.9, 0.01)
    y = wide.to(torch.bfloat16)[:, 1:4998]
    check(y, np.linspace(0, 0.99, 16, dtype=np.float32), 0.9, 0, 0.9, 0.0)
    n = 16
    f = torch.full((n,), 0.9, device="cuda")
    k = torch.full((n,), 50, dtype=torch.int32, device="cuda")
    u, mp = torch.rand(n, device="cuda"), torch.zeros(n, device="cuda")
    buf = torch.randn(n, 70000, device="cuda")
    q3.sample_given(buf, u, f, k, f, mp)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ids, lp = q3.sample_given(buf, u, f, k, f, mp)
    for _ in range(3):
        buf.normal_()
        u.uniform_()
        gr.replay()
        want, wlp = q3.sample_given(buf, u, f, k, f, mp)
        assert torch.equal(ids, want) and torch.equal(lp, wlp)


def test_share_of_the_kept_weight():
    """The ids of evenly spread u have the shares of their weights: a row of 64 ids, 4096 draws."""
    import speech_lm_decode_gb300 as q3
    x = torch.randn(64, generator=torch.Generator().manual_seed(5)) * 2
    n = 4096
    rows = x.cuda().expand(n, 64).contiguous()
    u = ((torch.arange(n) + 0.5) / n).cuda()
    one = torch.ones(n, device="cuda")
    ids, lp = q3.sample_given(rows, u, one, torch.zeros(n, dtype=torch.int32, device="cuda"), one, 0 * one)
    share = torch.softmax(x.double(), 0)
    count = torch.bincount(ids.cpu().long(), minlength=64).double() / n
    # a grid of n points meets an interval of length s between n s - 1 and n s + 1 times
    assert (count - share).abs().max() <= 1.0 / n + 1e-6
    assert (lp.cpu().double() - share.log()[ids.cpu().long()]).abs().max() < 1e-5


def test_refusals():
    import speech_lm_decode_gb300 as q3
    x = torch.randn(2, 100, device="cuda")
    f = torch.ones(2, device="cuda")
    k = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (x.half(), x.cpu(), x[0], x.t(), x[:1].expand(2, 100)):
        with pytest.raises(ValueError):
            q3.sample_given(bad, f, f, k, f, f)
    with pytest.raises(ValueError):
        q3.sample_given(x, f[:1], f, k, f, f)
    with pytest.raises(ValueError):
        q3.sample_given(x, f, f, k.long(), f, f)
    with pytest.raises(q3.Q3Error):
        q3.sample_given(torch.zeros(1, 262145, device="cuda"), f[:1], f[:1], k[:1], f[:1], f[:1])
    ids, lp = q3.sample_given(x[:0], f[:0], f[:0], k[:0], f[:0], f[:0])
    assert ids.shape == (0,) and lp.shape == (0,)
