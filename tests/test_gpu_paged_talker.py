"""The talker over a paged cache (kv_page_size > 0): the same parity with the oracle as over slabs."""
import ctypes
import dataclasses

import numpy as np
import pytest

import synth
from synth import BF16, F32
from parity import compare, run_gpu
from test_gpu_parity import small_weights, small_workload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims,dtype", [(synth.DIMS_SMALL, F32), (synth.DIMS_SMALL, BF16), (synth.DIMS_SMALL_PROJ, BF16)])
@pytest.mark.parametrize("pool", ["full", "exact"])
def test_parity_with_the_oracle(dims, dtype, pool):
    """Rows of unlike lengths; a pool of every position, or of exactly the pages that the rows need."""
    import speech_lm_decode_gb300 as q3
    wl = small_workload(dims, dtype)
    w = small_weights(wl)
    inp = synth.make_inputs(wl)
    pages = 0 if pool == "full" else sum(-(-(n + r.max_frames) // 16) for n, r in zip(wl.prompt_lens, wl.rows))
    g = run_gpu(wl, q3.to_device_weights(w), inp, cap_rows=list(range(wl.batch)), chunks=[4, 1, wl.frames - 5],
                expect_path=q3.Q3_PATH_GRAPH, kv_page_size=16, kv_pages=pages)
    assert g.frames[2] == 5 and g.reasons[2] == q3.Q3_FINISHED_EOS
    s = compare(wl, w, inp, g)
    assert s["checked"] > 0.5 * s["decisions"]


def test_one_row_and_longer_prompts():
    """Batch 1 (no frame kernel: the step runs per layer) and prompts that take the many-row attention kernel,
    against the oracle."""
    import speech_lm_decode_gb300 as q3
    for lens in ([150], [70, 1, 200]):
        wl = small_workload(synth.DIMS_SMALL, BF16, frames=6)
        wl = dataclasses.replace(wl, batch=len(lens), prompt_lens=lens, n_text=wl.n_text[:len(lens)],
                                 rows=[dataclasses.replace(r, max_frames=6) for r in wl.rows[:len(lens)]],
                                 max_ctx=max(lens) + 9)
        w = small_weights(wl)
        inp = synth.make_inputs(wl)
        g = run_gpu(wl, q3.to_device_weights(w), inp, cap_rows=list(range(wl.batch)), expect_path=q3.Q3_PATH_GRAPH,
                    kv_page_size=32)
        compare(wl, w, inp, g)


def test_second_prefill_and_capacity():
    import speech_lm_decode_gb300 as q3
    wl = small_workload(synth.DIMS_SMALL, BF16)
    w = small_weights(wl)
    inp = synth.make_inputs(wl)
    dw = q3.to_device_weights(w)
    need = sum(-(-(n + r.max_frames) // 16) for n, r in zip(wl.prompt_lens, wl.rows))
    args = (inp["prompt"], inp["prompt_offsets"], inp["text"], inp["text_offsets"], inp["tts_pad"], wl.rows)
    tts = q3.Q3TTS(wl.dims, BF16, dw, wl.batch, wl.max_ctx, max(wl.n_text), kv_page_size=16, kv_pages=need)
    try:
        a0 = tts.prefill(*args)
        a, _, _ = tts.step_frames(wl.frames)
        b0 = tts.prefill(*args)      # the pages are handed out anew
        b, _, _ = tts.step_frames(wl.frames)
        assert np.array_equal(a0, b0) and np.array_equal(a, b)
    finally:
        tts.close()
    tts = q3.Q3TTS(wl.dims, BF16, dw, wl.batch, wl.max_ctx, max(wl.n_text), kv_page_size=16, kv_pages=need - 1)
    try:
        rc, _ = tts.prefill(*args, check=False)
        assert rc == q3.Q3_ERR_CAPACITY
    finally:
        tts.close()
