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
