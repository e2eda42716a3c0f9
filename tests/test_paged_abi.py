"""The paged-cache header and its argument checks, on the CPU: nothing is queued when an argument is refused."""
import ctypes

import pytest

from test_abi import declared_symbols

ERR_ARG, ERR_CAPACITY = 1, 3


def cache(q3, **kw):
    c = q3.PagedCache()
    base = dict(n_q_heads=16, n_kv_heads=8, head_dim=128, act_dtype=q3.Q3_F32, kv_dtype=q3.Q3_BF16, page_size=16,
                n_pages=4, n_seqs=2, max_pages=3, k_pages=4096, v_pages=8192, page_table=256)
    for k, v in {**base, **kw}.items():
        setattr(c, k, v)
    return c


def test_exports():
    import speech_lm_decode_gb300 as q3
    names = declared_symbols("q3paged.h", "q3paged_")
    assert set(names) == set(q3.PAGED_EXPORTS)
    lib = q3.lib()
    assert all(hasattr(lib, n) for n in names) and hasattr(lib, "q3tts_sample_given")


BAD = [dict(head_dim=64), dict(n_q_heads=12), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_q_heads=34, n_kv_heads=2),
       dict(page_size=0), dict(page_size=8), dict(page_size=24), dict(page_size=2048), dict(n_pages=0), dict(n_seqs=0),
       dict(max_pages=0), dict(max_pages=1 << 30), dict(act_dtype=2), dict(kv_dtype=-1), dict(act_dtype=1, kv_dtype=0)]


@pytest.mark.parametrize("kw", BAD, ids=lambda kw: "-".join(f"{k}={v}" for k, v in kw.items()))
def test_caches_that_are_refused(kw):
    import speech_lm_decode_gb300 as q3
    L = q3.lib()
    c = cache(q3, **kw)
    assert L.q3paged_workspace_bytes(ctypes.byref(c)) == 0
    assert L.q3paged_append(ctypes.byref(c), 1, 4096, 0, 256, 256, None, None, 1e-6, 4096, 8, 4096, 0, None, None) == ERR_ARG
    assert L.q3paged_last_error()


def test_arguments_that_are_refused():
    import speech_lm_decode_gb300 as q3
    L = q3.lib()
    ok = cache(q3)
    ws = L.q3paged_workspace_bytes(ctypes.byref(ok))
    assert ws > 0 and ws == L.q3paged_workspace_bytes(ctypes.byref(cache(q3, act_dtype=q3.Q3_BF16)))

    def append(c=ok, n=1, qkv=4096, ld=0, seq=256, pos=256, qn=None, kn=None, eps=1e-6, rope=4096, rows=8, out=4096, ldo=0):
        return L.q3paged_append(ctypes.byref(c), n, qkv, ld, seq, pos, qn, kn, eps, rope, rows, out, ldo, None, None)

    def attend(c=ok, n=1, max_q=1, q=4096, ld=0, off=256, ctx=256, scale=0.1, out=4096, ldo=0, w=4096, wb=ws):
        return L.q3paged_attention(ctypes.byref(c), n, max_q, q, ld, off, ctx, scale, out, ldo, w, wb, None, None)
    for kw in (dict(n=-1), dict(qkv=None), dict(qkv=4100), dict(ld=100), dict(ld=4097), dict(seq=None), dict(pos=None),
               dict(qn=4096), dict(kn=4096), dict(qn=4100, kn=4096), dict(eps=-1.0), dict(eps=float("nan")),
               dict(rope=None), dict(rope=4100), dict(rows=0), dict(out=None), dict(ldo=64)):
        assert append(**kw) == ERR_ARG, kw
    for kw in (dict(n=-1), dict(max_q=-1), dict(q=None), dict(q=4104), dict(ld=2), dict(off=None), dict(ctx=None),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(out=None),
               dict(out=4104), dict(w=None), dict(w=4100)):
        assert attend(**kw) == ERR_ARG, kw
    assert attend(wb=ws - 1) == ERR_CAPACITY
    for kw in (dict(k_pages=None), dict(v_pages=4100), dict(page_table=None), dict(token_stride=64),
               dict(head_stride=129), dict(page_stride=-8), dict(page_stride=1 << 60)):
        assert append(cache(q3, **kw)) == ERR_ARG and attend(cache(q3, **kw)) == ERR_ARG, kw
    assert append(n=0) == 0 and attend(n=0) == 0 and attend(max_q=0) == 0
    assert L.q3paged_append(None, 1, 4096, 0, 256, 256, None, None, 1e-6, 4096, 8, 4096, 0, None, None) == ERR_ARG

    def draw(n=1, V=10, x=4096, dt=0, ld=0, u=256, t=256, k=256, p=256, mp=256, ids=256):
        return L.q3tts_sample_given(n, V, x, dt, ld, u, t, k, p, mp, ids, None, None, None)
    for kw in (dict(n=-1), dict(n=65536), dict(V=0), dict(V=262145), dict(dt=2), dict(x=None), dict(u=None),
               dict(t=None), dict(k=None), dict(p=None), dict(mp=None), dict(ids=None), dict(ld=9)):
        assert draw(**kw) == ERR_ARG, kw
    assert draw(n=0) == 0


def test_an_injected_timeout_is_not_negative():
    import speech_lm_decode_gb300 as q3
    L = q3.lib()
    assert L.q3paged_workspace_bytes(ctypes.byref(cache(q3, inject_timeout=3))) > 0
    assert L.q3paged_workspace_bytes(ctypes.byref(cache(q3, inject_timeout=-1))) == 0
    assert b"inject_timeout" in L.q3paged_last_error()
