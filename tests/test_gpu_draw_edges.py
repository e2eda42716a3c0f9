"""The draw from given numbers where little decides: borders within a step of a weight, histograms that fall short."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_ref import F, spec_exp  # noqa: E402
from test_gpu_draw_given import check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,vocab", [(40, 90000), (80, 50001), (20, 262144), (3, 30000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_histograms_that_fall_short_of_the_limit(n, vocab, dtype):
    """Crowds whose weights the histogram rounds down, by 2^-14 of them, under a top-p nearer to 1 than that: no bin
    of it reaches the limit, on any of a row's CTAs."""
    d = -np.arange(1, 400, dtype=np.float32) / 64       # (bf16 too)
    low = spec_exp(d).view(np.uint32) & 0x7FF
    d = d[(low > 0x300) & (low < 0x400)]
    rng = np.random.default_rng(n)
    x = np.empty((n, vocab), np.float32)
    for i in range(n):
        few = rng.choice(d, 1 + i % 3)
        x[i] = rng.choice(few, vocab)
        x[i, rng.integers(0, vocab, 2)] = 0
    x[n // 2, :5] = -np.inf
    p = rng.choice([0.99999, 0.999995, 0.9999999, 1 - 2.0 ** -24], n).astype(np.float32)
    u = rng.random(n).astype(np.float32)
    u[::3] = 1 - 2.0 ** -24
    check(torch.from_numpy(x).to(dtype).cuda(), u, 1.0, 0, p, 0.0)


def crowds(rows, vocab, dtype, seed):
    """Rows of two values, the smaller one where top-p cuts, with as many of the larger as bring the border nearest to a
    step between two ids: it comes out one id off where the weight of the smaller value is a step of fp32 off."""
    rng = np.random.default_rng(seed)
    x, p = np.empty((rows, vocab), np.float32), np.empty(rows, np.float32)
    one = 1 << 40
    near = []
    for i in range(rows):
        d = np.float32(torch.tensor(-rng.uniform(1.0, 2.3)).to(dtype).float())
        e = float(spec_exp(np.array([d], np.float32))[0])
        w = int(np.floor(np.ldexp(e, 40)))
        best = (1.0, 0, 0)
        top = np.arange(int(0.2 * e * vocab), int(0.4 * e * vocab), dtype=np.int64)
        for a in range(28, 44):
            # top-p a / 64 cuts at a / 64 of the whole weight: top + kept w, with how far that is from whole ids
            rest = (a * ((vocab - top) * w + top * one) - 64 * top * one) % (64 * w)
            off = np.minimum(rest, 64 * w - rest) / (64 * w)
            # against what a step of e, 2^-24 of it at least, moves the border by
            off = off / ((1 - a / 64) * top / e * 2.0 ** -24)
            best = min(best, (off.min(), a, int(top[off.argmin()])))
        near.append(best[0])
        p[i] = best[1] / 64
        x[i] = d
        x[i, rng.choice(vocab, best[2], replace=False)] = 0
    assert np.median(near) < 0.5
    return torch.from_numpy(x).to(dtype), rng.random(rows).astype(np.float32), p


# in shared memory, by a cluster and by one CTA; read again from L2, by one and by two CTAs
@pytest.mark.parametrize("rows,vocab", [(30, 40000), (150, 15000), (160, 60000), (80, 60000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_borders_within_a_step_of_a_weight(rows, vocab, dtype):
    x, u, p = crowds(rows, vocab, dtype, vocab)
    check(x.cuda(), u, 1.0, 0, p, 0.0)
