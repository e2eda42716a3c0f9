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
