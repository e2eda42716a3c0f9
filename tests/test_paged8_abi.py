"""The 8-bit cache's header and its argument checks, and those of the logits processors, on the CPU: nothing is queued
when an argument is refused."""
import ctypes

import pytest

from test_abi import declared_symbols

ERR_ARG, ERR_CAPACITY = 1, 3


def cache(q3, **kw):
    c = q3.Paged8Cache()
    base = dict(n_q_heads=16, n_kv_heads=8, head_dim=128, act_dtype=q3.Q3_F32, kv_dtype=q3.Q3_E4M3, page_size=32,
                n_pages=4, n_seqs=2, max_pages=3, k_pages=4096, v_pages=8192, page_table=256, scale_block=16, k_scale=64,
                v_scale=65)
    for k, v in {**base, **kw}.items():
        setattr(c if k in ("scale_block", "k_scale", "v_scale") else c.cache, k, v)
    return c


def test_exports():
    import speech_lm_decode_gb300 as q3
    names = declared_symbols("q3paged8.h", "q3paged8_")
    assert set(names) == set(q3.PAGED8_EXPORTS)
    lib = q3.lib()
    assert all(hasattr(lib, n) for n in names) and hasattr(lib, "q3tts_process_logits")


BAD = [dict(head_dim=64), dict(n_q_heads=12), dict(n_kv_heads=0), dict(n_q_heads=34, n_kv_heads=2), dict(page_size=0),
       dict(page_size=8), dict(page_size=24), dict(page_size=2048), dict(n_pages=0), dict(n_seqs=0), dict(max_pages=0),
       dict(max_pages=1 << 30), dict(act_dtype=2), dict(kv_dtype=0), dict(kv_dtype=1), dict(kv_dtype=3), dict(scale_block=0),
       dict(scale_block=8), dict(scale_block=24), dict(scale_block=64), dict(scale_block=-16), dict(inject_timeout=-1)]


@pytest.mark.parametrize("kw", BAD, ids=lambda kw: "-".join(f"{k}={v}" for k, v in kw.items()))
def test_caches_that_are_refused(kw):
    import speech_lm_decode_gb300 as q3
    L = q3.lib()
    c = ctypes.byref(cache(q3, **kw))
    assert L.q3paged8_workspace_bytes(c) == 0
    assert L.q3paged8_append(c, 1, 1, 4096, 0, 256, 256, None, None, 1e-6, 4096, 8, 4096, 0, None, None) == ERR_ARG
    assert L.q3paged8_attention(c, 1, 1, 4096, 0, 256, 256, 0.1, 4096, 0, 4096, 1 << 40, None, None) == ERR_ARG
    assert L.q3paged8_read(c, 1, 256, 0, 4096, 4096, None, None) == ERR_ARG
    assert L.q3paged_last_error()


def test_the_other_cache_takes_no_codes():
    import speech_lm_decode_gb300 as q3
    c = cache(q3).cache
    assert q3.lib().q3paged_workspace_bytes(ctypes.byref(c)) == 0


def test_arguments_that_are_refused():
    import speech_lm_decode_gb300 as q3
    L = q3.lib()
    ok = cache(q3)
    ws = L.q3paged8_workspace_bytes(ctypes.byref(ok))
    assert ws > 0 and ws == L.q3paged8_workspace_bytes(ctypes.byref(cache(q3, act_dtype=q3.Q3_BF16)))

    def append(c=ok, n=1, max_q=1, qkv=4096, ld=0, off=256, ctx=256, qn=None, kn=None, eps=1e-6, rope=4096, rows=8, out=4096, ldo=0):
        return L.q3paged8_append(ctypes.byref(c), n, max_q, qkv, ld, off, ctx, qn, kn, eps, rope, rows, out, ldo, None, None)

    def attend(c=ok, n=1, max_q=1, q=4096, ld=0, off=256, ctx=256, scale=0.1, out=4096, ldo=0, w=4096, wb=ws):
        return L.q3paged8_attention(ctypes.byref(c), n, max_q, q, ld, off, ctx, scale, out, ldo, w, wb, None, None)

    def read(c=ok, n=1, pages=256, dt=0, k=4096, v=4096):
        return L.q3paged8_read(ctypes.byref(c), n, pages, dt, k, v, None, None)
    for kw in (dict(n=-1), dict(max_q=-1), dict(qkv=None), dict(qkv=4100), dict(ld=100), dict(ld=4097), dict(off=None),
               dict(ctx=None), dict(qn=4096), dict(kn=4096), dict(qn=4100, kn=4096), dict(eps=-1.0), dict(eps=float("nan")),
               dict(rope=None), dict(rope=4100), dict(rows=0), dict(out=None), dict(ldo=64)):
        assert append(**kw) == ERR_ARG, kw
    for kw in (dict(n=-1), dict(max_q=-1), dict(q=None), dict(q=4104), dict(ld=2), dict(off=None), dict(ctx=None),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(out=None),
               dict(out=4104), dict(w=None), dict(w=4100)):
        assert attend(**kw) == ERR_ARG, kw
    assert attend(wb=ws - 1) == ERR_CAPACITY
    for kw in (dict(n=-1), dict(pages=None), dict(dt=2), dict(k=4100), dict(v=4104)):
        assert read(**kw) == ERR_ARG, kw
    for kw in (dict(k_pages=None), dict(v_pages=4100), dict(page_table=None), dict(token_stride=64), dict(head_stride=129),
               dict(page_stride=-16), dict(page_stride=1 << 60), dict(token_stride=1 << 26), dict(k_scale=None), dict(v_scale=None)):
        c = cache(q3, **kw)
        assert append(c) == ERR_ARG and attend(c) == ERR_ARG and read(c) == ERR_ARG, kw
    assert append(n=0) == 0 and append(max_q=0) == 0 and attend(n=0) == 0 and attend(max_q=0) == 0
    assert read(n=0) == 0 and read(k=None, v=None) == 0
    assert L.q3paged8_append(None, 1, 1, 4096, 0, 256, 256, None, None, 1e-6, 4096, 8, 4096, 0, None, None) == ERR_ARG


def test_logits_arguments_that_are_refused():
    import speech_lm_decode_gb300 as q3
    L = q3.lib()

    def process(n=1, V=100, x=4096, dt=0, ld=0, h=256, cap=10, ldh=0, nh=256, np_=256, rep=256, pres=256, freq=256, nb=3,
                bo=256, bi=256, b=256, nm=1, m=256, ldm=0, mr=256, out=8192, ldo=0):
        return L.q3tts_process_logits(n, V, x, dt, ld, h, cap, ldh, nh, np_, rep, pres, freq, nb, bo, bi, b, nm, m, ldm, mr,
                                      out, ldo, None, None)
    for kw in (dict(n=-1), dict(n=65536), dict(V=0), dict(V=262145), dict(dt=2), dict(x=None), dict(out=None), dict(ld=99),
               dict(ldo=99), dict(x=4096, out=4096, ld=100, ldo=101), dict(h=None), dict(nh=None), dict(cap=-1),
               dict(cap=(1 << 28) + 1), dict(ldh=9), dict(bo=None), dict(bi=None), dict(b=None), dict(nb=-1), dict(nm=0),
               dict(mr=None, n=2), dict(m=None), dict(ldm=3)):
        assert process(**kw) == ERR_ARG, kw
        assert L.q3paged_last_error()
    assert process(n=0) == 0
