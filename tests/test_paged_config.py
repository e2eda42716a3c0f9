"""The paged cache's config fields (CPU only)."""
import ctypes


def test_fields_are_validated_and_size_the_pool():
    import speech_lm_decode_gb300 as q3
    import synth
    L = q3.lib()

    def size(batch=32, **kw):
        c = q3.make_config(synth.DIMS_06B, q3.Q3_BF16, batch, 768, 64, **kw)
        return L.q3tts_workspace_bytes(ctypes.byref(c))
    slabs = size()
    for kw in ({"kv_page_size": 8}, {"kv_page_size": 24}, {"kv_page_size": 2048}, {"kv_page_size": -16},
               {"kv_pages": 5}, {"kv_page_size": 16, "kv_pages": -1},
               {"kv_page_size": 16, "step_path": q3.Q3_PATH_FRAME}, {"kv_page_size": 16, "step_path": q3.Q3_PATH_CLUSTER}):
        assert size(**kw) == 0, kw
    position = 28 * 8 * 128 * 2 * 2      # layers x heads x values x K and V x bytes
    full = size(kv_page_size=16)
    assert size(kv_page_size=16, kv_pages=32 * 48) == full and full >= slabs
    half = size(kv_page_size=16, kv_pages=16 * 48)
    assert abs((full - half) - 16 * 768 * position) <= 4096
    assert size(batch=1, kv_page_size=64) > 0
