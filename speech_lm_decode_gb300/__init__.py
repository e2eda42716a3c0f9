"""GB300 (sm_103a) Qwen3-TTS 12 Hz frame loop: Python binding of libq3tts.so.

Argument marshalling only: every step of the frame loop runs in the library's
CUDA kernels.  PyTorch provides device memory and the stream.  The library
must have been built (``speech_lm_decode_gb300.build.build()``); importing the
binding without it raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import weakref

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq3tts.so")

Q3_OK, Q3_ERR_ARG, Q3_ERR_CUDA, Q3_ERR_CAPACITY, Q3_ERR_STATE, Q3_ERR_NAN, Q3_ERR_TIMEOUT, Q3_ERR_BOUNDS = range(8)
Q3_F32, Q3_BF16 = 0, 1
Q3_RUNNING, Q3_FINISHED_EOS, Q3_FINISHED_LENGTH, Q3_FINISHED_ERROR = 0, 1, 2, 3
Q3_PATH_AUTO, Q3_PATH_GRAPH, Q3_PATH_FRAME, Q3_PATH_CLUSTER = 0, 1, 2, 3
PATH_NAMES = {Q3_PATH_GRAPH: "graph", Q3_PATH_FRAME: "frame", Q3_PATH_CLUSTER: "cluster"}

EXPORTS = ("q3tts_workspace_bytes", "q3tts_create", "q3tts_prefill", "q3tts_step_frames", "q3tts_set_capture",
           "q3tts_sample_logits", "q3tts_sample_logits_noalloc", "q3tts_step_kernel_count", "q3tts_step_path",
           "q3tts_text_embed", "q3tts_sample_given", "q3tts_last_error", "q3tts_destroy")


class Q3Error(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"q3tts error {code}: {msg}")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim", "ffn",
                                            "codec_vocab", "cp_layers", "cp_hidden", "cp_ffn", "cp_vocab",
                                            "n_groups", "eos_id", "suppress_lo", "suppress_hi")] + \
              [("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float)] + \
              [(n, ctypes.c_int) for n in ("dtype", "max_batch", "max_ctx", "max_text", "step_path", "tc_min_tokens",
                                           "debug_sync", "wait_limit_us", "inject_timeout", "text_vocab",
                                           "text_hidden", "separate_projections", "kv_page_size", "kv_pages")]

# execution fields of the config (everything else comes from the model dims)
EXEC_FIELDS = ("step_path", "tc_min_tokens", "debug_sync", "wait_limit_us", "inject_timeout",
               "separate_projections", "kv_page_size", "kv_pages")


class BlockWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("attn_norm", "wqkv", "q_norm", "k_norm", "wo", "mlp_norm", "wgu",
                                               "wd", "final_norm")]


class Weights(ctypes.Structure):
    _fields_ = [("talker", BlockWeights), ("codec_emb", ctypes.c_void_p), ("codec_head", ctypes.c_void_p),
                ("cp", BlockWeights), ("cp_emb", ctypes.c_void_p), ("cp_heads", ctypes.c_void_p),
                ("cp_proj_w", ctypes.c_void_p), ("cp_proj_b", ctypes.c_void_p)] + \
              [(n, ctypes.c_void_p) for n in ("text_emb", "text_fc1_w", "text_fc1_b", "text_fc2_w", "text_fc2_b")]

TEXT_KEYS = ("text_emb", "text_fc1_w", "text_fc1_b", "text_fc2_w", "text_fc2_b")


class Sampling(ctypes.Structure):
    _fields_ = [("do_sample", ctypes.c_int), ("temperature", ctypes.c_float), ("top_k", ctypes.c_int),
                ("top_p", ctypes.c_float), ("repetition_penalty", ctypes.c_float), ("min_new_tokens", ctypes.c_int),
                ("seed", ctypes.c_uint64), ("max_frames", ctypes.c_int), ("force_eos_at_frame", ctypes.c_int),
                ("cp_do_sample", ctypes.c_int), ("cp_temperature", ctypes.c_float), ("cp_top_k", ctypes.c_int),
                ("cp_top_p", ctypes.c_float)]


_lib = None


def lib():
    """The loaded libq3tts.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with speech_lm_decode_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        L.q3tts_workspace_bytes.restype = ctypes.c_size_t
        L.q3tts_workspace_bytes.argtypes = [ctypes.POINTER(Config)]
        L.q3tts_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), vp, ctypes.c_size_t, vp,
                                   ctypes.POINTER(vp)]
        L.q3tts_prefill.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp]
        L.q3tts_step_frames.argtypes = [vp, i32, vp, vp, vp]
        L.q3tts_set_capture.argtypes = [vp, i32, vp, vp, vp, i32]
        L.q3tts_sample_logits.argtypes = [vp, i32, vp, i32, vp, vp, vp, i32, vp, vp]
        L.q3tts_step_kernel_count.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
        L.q3tts_step_path.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_int)]
        L.q3tts_text_embed.argtypes = [vp, i32, vp, vp]
        L.q3tts_sample_logits_noalloc.argtypes = [i32, i32, vp, i32, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp]
        i64, f32 = ctypes.c_int64, ctypes.c_float
        L.q3tts_sample_given.argtypes = [i32, i32, vp, i32, i64] + [vp] * 9
        L.q3paged_append.argtypes = [vp, i32, vp, i64, vp, vp, vp, vp, f32, vp, i32, vp, i64, vp, vp]
        L.q3paged_workspace_bytes.restype = ctypes.c_size_t
        L.q3paged_workspace_bytes.argtypes = [vp]
        L.q3paged_attention.argtypes = [vp, i32, i32, vp, i64, vp, vp, f32, vp, i64, vp, ctypes.c_size_t, vp, vp]
        L.q3paged_last_error.restype = ctypes.c_char_p
        L.q3paged_last_error.argtypes = []
        L.q3tts_last_error.restype = ctypes.c_char_p
        L.q3tts_last_error.argtypes = [vp]
        L.q3tts_destroy.argtypes = [vp]
        _lib = L
    return _lib


def make_config(dims, dtype: int, max_batch: int, max_ctx: int, max_text: int, **exec_opts) -> Config:
    """exec_opts: step_path, tc_min_tokens, debug_sync, wait_limit_us, inject_timeout,
    separate_projections, kv_page_size, kv_pages (default 0)."""
    unknown = set(exec_opts) - set(EXEC_FIELDS)
    if unknown:
        raise ValueError(f"unknown config options {sorted(unknown)}")
    c = Config()
    for f, _ in Config._fields_:
        if f in EXEC_FIELDS:
            setattr(c, f, int(exec_opts.get(f, 0)))
        elif f == "dtype":
            c.dtype = dtype
        elif f == "max_batch":
            c.max_batch = max_batch
        elif f == "max_ctx":
            c.max_ctx = max_ctx
        elif f == "max_text":
            c.max_text = max_text
        else:
            setattr(c, f, getattr(dims, f, 0))
    return c


def make_sampling(r) -> Sampling:
    s = Sampling()
    for f, _ in Sampling._fields_:
        setattr(s, f, getattr(r, f))
    return s


def to_device_weights(w: dict, device="cuda") -> dict:
    """Host weight arrays (bf16 as uint16 bit patterns) -> device tensors of the same layout."""
    import torch

    def dev(a):
        if a is None:
            return None
        t = torch.from_numpy(np.ascontiguousarray(a))
        if a.dtype == np.uint16:
            t = t.view(torch.bfloat16)
        return t.to(device)
    out = {}
    for k, v in w.items():
        out[k] = {kk: dev(vv) for kk, vv in v.items()} if isinstance(v, dict) else dev(v)
    return out


def _ptr(t):
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data


def make_weights(dw: dict) -> Weights:
    ws = Weights()
    for blk in ("talker", "cp"):
        b = getattr(ws, blk)
        for k, _ in BlockWeights._fields_:
            setattr(b, k, _ptr(dw[blk][k]))
    for k in ("codec_emb", "codec_head", "cp_emb", "cp_heads", "cp_proj_w", "cp_proj_b") + TEXT_KEYS:
        setattr(ws, k, _ptr(dw.get(k)))
    return ws


class Q3TTS:
    """One handle: model weights (borrowed device tensors), a workspace and a stream."""

    def __init__(self, dims, dtype: int, device_weights: dict, max_batch: int, max_ctx: int, max_text: int,
                 stream=None, **exec_opts):
        import torch
        self._dw = device_weights
        self.dims, self.dtype = dims, dtype
        self.cfg = make_config(dims, dtype, max_batch, max_ctx, max_text, **exec_opts)
        nbytes = lib().q3tts_workspace_bytes(ctypes.byref(self.cfg))
        if nbytes == 0:
            raise Q3Error(Q3_ERR_ARG, "invalid configuration")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        self._w = make_weights(device_weights)
        h = ctypes.c_void_p()
        rc = lib().q3tts_create(ctypes.byref(self.cfg), ctypes.byref(self._w), self.workspace.data_ptr(), nbytes,
                                self.stream.cuda_stream, ctypes.byref(h))
        if rc:
            raise Q3Error(rc, "q3tts_create failed")
        self.h = h.value
        self.batch = 0

    def _check(self, rc):
        if rc:
            raise Q3Error(rc, lib().q3tts_last_error(self.h).decode())

    def close(self):
        if getattr(self, "h", None):
            lib().q3tts_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, prompt, prompt_offsets, text, text_offsets, tts_pad, rows, check=True):
        """prompt/text/tts_pad: fp32 numpy arrays or torch tensors (host or cuda)."""
        B = len(rows)
        po = np.ascontiguousarray(prompt_offsets, dtype=np.int32)
        to = np.ascontiguousarray(text_offsets, dtype=np.int32)
        sp = (Sampling * B)(*[make_sampling(r) for r in rows])
        keep = [prompt, text, tts_pad]
        code0 = np.full(B, -1, np.int32)
        rc = lib().q3tts_prefill(self.h, B, _ptr(prompt), po.ctypes.data,
                                 _ptr(text) if text is not None and len(text) else None, to.ctypes.data,
                                 _ptr(tts_pad), ctypes.cast(sp, ctypes.c_void_p), code0.ctypes.data)
        del keep
        if check:
            self._check(rc)
        self.batch = B
        return code0 if check else (rc, code0)

    def step_frames(self, n: int, codes_out=None, check=True):
        """Run n talker steps.  codes_out: None (host numpy returned), or a
        [B, n, G] int32 numpy array / torch tensor to fill."""
        B, G = self.batch, self.dims.n_groups
        out = np.empty((B, n, G), np.int32) if codes_out is None else codes_out
        frames = np.zeros(B, np.int32)
        reasons = np.zeros(B, np.int32)
        rc = lib().q3tts_step_frames(self.h, n, _ptr(out), frames.ctypes.data, reasons.ctypes.data)
        if check:
            self._check(rc)
            return out, frames, reasons
        return rc, out, frames, reasons

    def text_embed(self, ids, out=None, check=True):
        """Talker-width rows of text token ids (gather + ResizeMLP on the GPU).
        ids: int32 numpy array or torch tensor (host or cuda); out: None (host
        numpy returned) or an [n, hidden] float32 array / tensor to fill."""
        n = int(len(ids))
        if isinstance(ids, np.ndarray) or not hasattr(ids, "data_ptr"):
            ids = np.ascontiguousarray(ids, dtype=np.int32)
        rows = np.empty((n, self.dims.hidden), np.float32) if out is None else out
        rc = lib().q3tts_text_embed(self.h, n, _ptr(ids) if n else None, _ptr(rows) if n else None)
        if check:
            self._check(rc)
            return rows
        return rc, rows

    def step_path(self, batch: int) -> int:
        """Q3_PATH_CLUSTER / Q3_PATH_FRAME / Q3_PATH_GRAPH: what runs a step of `batch` rows."""
        p = ctypes.c_int(0)
        self._check(lib().q3tts_step_path(self.h, batch, ctypes.byref(p)))
        return p.value

    def step_kernel_count(self) -> int:
        n = ctypes.c_int(0)
        self._check(lib().q3tts_step_kernel_count(self.h, ctypes.byref(n)))
        return n.value

    def set_capture(self, rows, talker_logits=None, cp_logits=None, max_frames=0):
        r = np.ascontiguousarray(rows, dtype=np.int32)
        self._cap = (r, talker_logits, cp_logits)
        self._check(lib().q3tts_set_capture(self.h, len(r), r.ctypes.data if len(r) else None, _ptr(talker_logits),
                                            _ptr(cp_logits), max_frames))

    def sample_logits(self, logits, talker: bool, params, sel_index, step: int, noise_row, seen=None, check=True):
        """Processors + draw on [n, V] fp32 logits (numpy or torch, host or cuda) -> ids [n]."""
        n = len(params)
        sp = (Sampling * n)(*[make_sampling(r) for r in params])
        sel = np.ascontiguousarray(sel_index, dtype=np.int32)
        nr = np.ascontiguousarray(noise_row, dtype=np.int32)
        if isinstance(logits, np.ndarray):
            logits = np.ascontiguousarray(logits, dtype=np.float32)
        if isinstance(seen, np.ndarray):
            seen = np.ascontiguousarray(seen, dtype=np.uint8)
        ids = np.full(n, -1, np.int32)
        rc = lib().q3tts_sample_logits(self.h, n, _ptr(logits), int(talker), ctypes.cast(sp, ctypes.c_void_p),
                                       _ptr(seen), sel.ctypes.data, step, nr.ctypes.data, ids.ctypes.data)
        if check:
            self._check(rc)
            return ids
        return rc, ids


def sample_logits_noalloc(logits, talker: bool, params, sel_index, step: int, noise_row, eos_id: int,
                          suppress_lo: int, suppress_hi: int, seen=None, stream=None, check=True):
    """Processors + draw without a handle or any device allocation.

    For callers that cannot allocate device memory: logits ([n, V] fp32) and
    seen ([n, V] uint8, optional) must already be CUDA tensors.  Returns the
    ids (host numpy).  Calls that overlap on the GPU race (one shared staging
    area per device)."""
    import torch
    # the library reads n * V * 4 bytes at logits and n * V at seen on the GPU,
    # and n entries of each host array: check all of it before passing pointers
    if not (isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dtype == torch.float32 and
            logits.dim() == 2 and logits.is_contiguous()):
        raise ValueError("logits must be a contiguous 2-D float32 CUDA tensor")
    n, V = int(logits.shape[0]), int(logits.shape[1])
    if seen is not None and not (isinstance(seen, torch.Tensor) and seen.is_cuda and seen.dtype == torch.uint8 and
                                 seen.is_contiguous() and tuple(seen.shape) == (n, V)):
        raise ValueError("seen must be None or a contiguous [n, V] uint8 CUDA tensor")
    sel = np.ascontiguousarray(sel_index, dtype=np.int32)
    nr = np.ascontiguousarray(noise_row, dtype=np.int32)
    if len(params) != n or sel.shape != (n,) or nr.shape != (n,):
        raise ValueError("params, sel_index and noise_row must have one entry per logit set")
    sp = (Sampling * max(n, 1))(*[make_sampling(r) for r in params])
    ids = np.full(max(n, 1), -1, np.int32)
    st = None if stream is None else stream.cuda_stream
    rc = lib().q3tts_sample_logits_noalloc(n, V, _ptr(logits), int(talker), ctypes.cast(sp, ctypes.c_void_p),
                                           _ptr(seen), sel.ctypes.data, step, nr.ctypes.data, eos_id, suppress_lo,
                                           suppress_hi, ids.ctypes.data, st)
    if check and rc:
        raise Q3Error(rc, "q3tts_sample_logits_noalloc failed")
    return ids[:n] if check else (rc, ids[:n])


# ---------------------------------------------------------------- codec decoder (q3codec.h)
CODEC_EXPORTS = ("q3codec_workspace_bytes", "q3codec_create", "q3codec_samples_per_frame", "q3codec_decode_window",
                 "q3codec_decode", "q3codec_stream_reset", "q3codec_stream_push", "q3codec_window_kernel_count",
                 "q3codec_last_error", "q3codec_destroy")
CODEC_MAX_BLOCKS = 4


class CodecConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_codebooks", "codebook_size", "codebook_dim", "hidden", "n_layers",
                                            "n_heads", "head_dim", "ffn", "window")] + \
              [(n, ctypes.c_float) for n in ("rope_theta", "rms_eps", "ln_eps")] + \
              [(n, ctypes.c_int) for n in ("n_up", "up_ffn", "dac_channels", "n_blocks")] + \
              [("strides", ctypes.c_int * CODEC_MAX_BLOCKS)] + \
              [(n, ctypes.c_int) for n in ("dtype", "max_frames", "tc_min_tokens")]


CODEC_KEYS = ("codebooks", "proj_sem", "proj_ac", "attn_norm", "wqkv", "wo", "ls_attn", "mlp_norm", "wgu", "wd",
              "ls_mlp", "final_norm", "up_w", "up_b", "dw_w", "dw_b", "ln_w", "ln_b", "fc1_w", "fc1_b", "fc2_w",
              "fc2_b", "gamma", "in_w", "in_b")
CODEC_BLOCK_KEYS = ("snake_a", "snake_b", "tconv_w", "tconv_b")
CODEC_UNIT_KEYS = ("a1", "b1", "w1", "c1", "a2", "b2", "w2", "c2")


class CodecWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in CODEC_KEYS] + \
              [("blk", (ctypes.c_void_p * 4) * CODEC_MAX_BLOCKS),
               ("unit", ((ctypes.c_void_p * 8) * 3) * CODEC_MAX_BLOCKS)] + \
              [(n, ctypes.c_void_p) for n in ("out_a", "out_b", "out_w", "out_bias")]


def _codec_lib():
    L = lib()
    if not getattr(L, "_codec_ready", False):
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        L.q3codec_workspace_bytes.restype = ctypes.c_size_t
        L.q3codec_workspace_bytes.argtypes = [ctypes.POINTER(CodecConfig)]
        L.q3codec_create.argtypes = [ctypes.POINTER(CodecConfig), ctypes.POINTER(CodecWeights), vp, ctypes.c_size_t,
                                     vp, ctypes.POINTER(vp)]
        L.q3codec_samples_per_frame.argtypes = [vp]
        L.q3codec_decode_window.argtypes = [vp, vp, i32, i32, vp]
        L.q3codec_decode.argtypes = [vp, vp, i32, vp]
        L.q3codec_stream_reset.argtypes = [vp]
        L.q3codec_stream_push.argtypes = [vp, vp, i32, i32, vp, ctypes.c_long, ctypes.POINTER(ctypes.c_long)]
        L.q3codec_window_kernel_count.argtypes = [vp]
        L.q3codec_last_error.restype = ctypes.c_char_p
        L.q3codec_last_error.argtypes = [vp]
        L.q3codec_destroy.argtypes = [vp]
        L._codec_ready = True
    return L


def make_codec_config(dims, dtype: int, max_frames: int, tc_min_tokens: int = 0) -> CodecConfig:
    c = CodecConfig()
    for f, _ in CodecConfig._fields_:
        if f == "strides":
            for i, s in enumerate(dims.strides):
                c.strides[i] = s
        elif f == "n_blocks":
            c.n_blocks = len(dims.strides)
        elif f == "dtype":
            c.dtype = dtype
        elif f == "max_frames":
            c.max_frames = max_frames
        elif f == "tc_min_tokens":
            c.tc_min_tokens = tc_min_tokens
        else:
            setattr(c, f, getattr(dims, f))
    return c


def codec_to_device(w: dict, device="cuda") -> dict:
    """Host decoder weights (synth layout) -> device tensors of the same layout."""
    import torch

    def dev(a):
        t = torch.from_numpy(np.ascontiguousarray(a))
        if a.dtype == np.uint16:
            t = t.view(torch.bfloat16)
        return t.to(device)
    out = {k: dev(v) for k, v in w.items() if k != "blocks"}
    out["blocks"] = [{k: ([{kk: dev(vv) for kk, vv in u.items()} for u in v] if k == "units" else dev(v))
                      for k, v in b.items()} for b in w["blocks"]]
    return out


class Q3Codec:
    """Codec decoder handle: borrowed device weights, a workspace and a stream."""

    def __init__(self, dims, dtype: int, device_weights: dict, max_frames: int = 325, stream=None,
                 tc_min_tokens: int = 0):
        import torch
        if len(dims.strides) > CODEC_MAX_BLOCKS:
            raise ValueError("at most 4 vocoder blocks")
        self._dw = device_weights
        self.dims, self.dtype = dims, dtype
        self.cfg = make_codec_config(dims, dtype, max_frames, tc_min_tokens)
        L = _codec_lib()
        nbytes = L.q3codec_workspace_bytes(ctypes.byref(self.cfg))
        if nbytes == 0:
            raise Q3Error(Q3_ERR_ARG, "invalid codec configuration")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        w = CodecWeights()
        for k in CODEC_KEYS + ("out_a", "out_b", "out_w", "out_bias"):
            setattr(w, k, _ptr(device_weights[k]))
        for b, blk in enumerate(device_weights["blocks"]):
            for i, k in enumerate(CODEC_BLOCK_KEYS):
                w.blk[b][i] = _ptr(blk[k])
            for u, unit in enumerate(blk["units"]):
                for i, k in enumerate(CODEC_UNIT_KEYS):
                    w.unit[b][u][i] = _ptr(unit[k])
        self._w = w
        h = ctypes.c_void_p()
        rc = L.q3codec_create(ctypes.byref(self.cfg), ctypes.byref(w), self.workspace.data_ptr(), nbytes,
                              self.stream.cuda_stream, ctypes.byref(h))
        if rc:
            raise Q3Error(rc, "q3codec_create failed")
        self.h = h.value
        self.spf = L.q3codec_samples_per_frame(self.h)

    def _check(self, rc):
        if rc:
            raise Q3Error(rc, _codec_lib().q3codec_last_error(self.h).decode())

    def close(self):
        if getattr(self, "h", None):
            _codec_lib().q3codec_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _codes(self, codes):
        if hasattr(codes, "data_ptr"):
            return codes
        return np.ascontiguousarray(codes, dtype=np.int32)

    def decode_window(self, codes, keep_from: int = 0, out=None, check=True):
        """codes [T, n_codebooks] int32 (numpy or torch, host or cuda) -> samples of
        frames keep_from..T-1 (numpy float32 unless `out` is given)."""
        codes = self._codes(codes)
        T = int(codes.shape[0])
        wav = np.empty((T - keep_from) * self.spf, np.float32) if out is None else out
        rc = _codec_lib().q3codec_decode_window(self.h, _ptr(codes), T, keep_from, _ptr(wav))
        if check:
            self._check(rc)
            return wav
        return rc, wav

    def decode(self, codes, out=None, check=True):
        """A whole request on the 300/25 chunk grid."""
        codes = self._codes(codes)
        T = int(codes.shape[0])
        wav = np.empty(T * self.spf, np.float32) if out is None else out
        rc = _codec_lib().q3codec_decode(self.h, _ptr(codes), T, _ptr(wav))
        if check:
            self._check(rc)
            return wav
        return rc, wav

    def stream_reset(self):
        self._check(_codec_lib().q3codec_stream_reset(self.h))

    def stream_push(self, codes, final=False, capacity=None, check=True):
        """Append host codes [n, n_codebooks]; returns the samples sent by the
        decodes that became due (numpy float32, possibly empty)."""
        codes = np.ascontiguousarray(codes, dtype=np.int32).reshape(-1, self.dims.n_codebooks)
        n = codes.shape[0]
        cap = capacity if capacity is not None else (n + 2 * 325) * self.spf
        buf = np.empty(max(cap, 1), np.float32)
        got = ctypes.c_long(0)
        rc = _codec_lib().q3codec_stream_push(self.h, codes.ctypes.data if n else None, n, int(final),
                                              buf.ctypes.data, cap, ctypes.byref(got))
        if check:
            self._check(rc)
            return buf[:got.value]
        return rc, buf[:got.value]

    def kernel_count(self) -> int:
        return _codec_lib().q3codec_window_kernel_count(self.h)


# ---------------------------------------------------------------- paged cache (q3paged.h)
PAGED_EXPORTS = ("q3paged_append", "q3paged_workspace_bytes", "q3paged_attention", "q3paged_last_error")
Q3PAGED_ERR_BOUNDS, Q3PAGED_ERR_TIMEOUT, Q3PAGED_COUNTER_BYTES = 2, 4, 4096


class PagedCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_q_heads", "n_kv_heads", "head_dim", "act_dtype", "kv_dtype",
                                            "page_size", "n_pages", "n_seqs", "max_pages")] + \
              [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride")] + \
              [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "page_table")] + [("inject_timeout", ctypes.c_int)]


def _paged_raise(rc):
    raise Q3Error(rc, lib().q3paged_last_error().decode())


def _dtype_code(t):
    import torch
    code = {torch.float32: Q3_F32, torch.bfloat16: Q3_BF16}.get(t.dtype)
    if code is None:
        raise ValueError(f"float32 or bfloat16 expected, not {t.dtype}")
    return code


class _on_device:
    """The tensors' device made current for a call (nothing to do where it is already)."""

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        import torch
        self.prev = torch.cuda.current_device()
        torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        import torch
        torch.cuda.set_device(self.prev)


def _need(t, name, dtype, shape, device):
    """A contiguous CUDA tensor of this type, shape and device index (the kernels read it by its address)."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device} is expected")
    return t.data_ptr()


def _on_stream(device, call):
    """call(stream) with the tensors' device current, on its current stream."""
    from torch import _C
    if _C._cuda_getDevice() == device:
        rc = call(_C._cuda_getCurrentRawStream(device))
    else:
        with _on_device(device):
            rc = call(_C._cuda_getCurrentRawStream(device))
    if rc:
        _paged_raise(rc)


# attention workspaces by (device, stream): calls of one stream follow each other, whichever cache they are for
_paged_workspaces = weakref.WeakValueDictionary()


class PagedKV:
    """A paged key / value cache over tensors that the caller owns (q3paged.h).

    k_pages, v_pages: CUDA tensors [n_pages, n_kv_heads, page_size, 128], float32 or bfloat16, of the same
    strides (a permuted view of [n_pages, page_size, n_kv_heads, 128] serves as well); page_table: int32
    [n_seqs, max_pages].  The tensors may be written between calls (the table as sequences grow); their
    addresses are taken once, here.  Work is queued on the current stream; calls on different streams have
    a workspace each (51 MB, which the cache objects used on a stream share and the last of them gives back), and a
    call that is being captured gets one of its graph's own.  Keep the object as long as graphs that were captured
    with it are replayed.  inject_timeout is for tests (q3paged_cache)."""

    def __init__(self, k_pages, v_pages, page_table, n_q_heads: int, inject_timeout: int = 0):
        import torch
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 4 and t.shape[3] == 128 and
                    t.stride(3) == 1):
                raise ValueError(f"{name}: a CUDA tensor [n_pages, n_kv_heads, page_size, 128] with contiguous rows "
                                 "is expected")
        if k_pages.dtype != v_pages.dtype or k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride() \
                or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must agree in type, shape, strides and device")
        if not (isinstance(page_table, torch.Tensor) and page_table.dim() == 2):
            raise ValueError("page_table: an int32 tensor [n_seqs, max_pages] is expected")
        self.device, self._dev = k_pages.device, k_pages.get_device()
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        c = PagedCache()
        c.n_pages, c.n_kv_heads, c.page_size, c.head_dim = k_pages.shape
        # 0 stands for packed: of an axis of one entry, whatever the tensor says
        steps = [st if size > 1 else 0 for size, st in zip(k_pages.shape[:3], k_pages.stride())]
        if any(size > 1 and st < 128 for size, st in zip(k_pages.shape[:3], steps)):
            raise ValueError("k_pages and v_pages: pages, heads and positions must not share memory")
        c.page_stride, c.head_stride, c.token_stride = steps
        c.n_q_heads, c.inject_timeout = n_q_heads, inject_timeout
        c.kv_dtype = _dtype_code(k_pages)
        c.n_seqs, c.max_pages = page_table.shape
        c.k_pages, c.v_pages = k_pages.data_ptr(), v_pages.data_ptr()
        c.page_table = _need(page_table, "page_table", torch.int32, page_table.shape, self._dev)
        self.nq, self.nkv = n_q_heads, c.n_kv_heads
        self._q_off_shape, self._ctx_shape = (c.n_seqs + 1,), (c.n_seqs,)
        # one description for each type of activations
        self._c = {}
        for act in (Q3_F32, Q3_BF16):
            d = PagedCache.from_buffer_copy(c)
            d.act_dtype = act
            self._c[torch.float32 if act == Q3_F32 else torch.bfloat16] = (d, ctypes.addressof(d))
        self._lib = lib()
        self.ws_bytes = self._lib.q3paged_workspace_bytes(self._c[torch.float32][1])
        if self.ws_bytes == 0:
            _paged_raise(Q3_ERR_ARG)
        self._ws = {}
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._err = self.err.data_ptr()

    def _workspace(self, stream):
        import torch
        if torch._C._cuda_isCurrentStreamCapturing():
            # the graph's own; a node of it clears the counters
            ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
            ws[:Q3PAGED_COUNTER_BYTES].zero_()
            return ws
        ws = self._ws.get(stream)
        if ws is None:
            ws = _paged_workspaces.get((self._dev, stream))
            if ws is None:
                ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)
                _paged_workspaces[self._dev, stream] = ws
            self._ws[stream] = ws
        return ws

    def _rows(self, t, name, heads, dtype=None):
        """A 2-D or 3-D CUDA tensor whose rows are heads * 128 contiguous values: (type, rows, row stride)."""
        shape, stride, width = t.shape, t.stride(), heads * 128
        if t.get_device() != self._dev or (dtype is not None and t.dtype is not dtype):
            raise ValueError(f"{name}: a tensor of the activations' type on {self.device} is expected")
        n = len(shape)
        if not ((n == 3 and shape[1] == heads and shape[2] == 128 and stride[2] == 1 and (heads == 1 or stride[1] == 128))
                or (n == 2 and shape[1] == width and stride[1] == 1)):
            raise ValueError(f"{name}: rows of {width} contiguous values are expected")
        if shape[0] > 1 and stride[0] < width:
            raise ValueError(f"{name}: rows must not share memory")
        return shape[0], (stride[0] if shape[0] > 1 else width)

    def _act(self, t):
        c = self._c.get(t.dtype)
        if c is None:
            raise ValueError(f"float32 or bfloat16 expected, not {t.dtype}")
        return c[1]

    def _out(self, out, n, like):
        import torch
        if out is None:
            return torch.empty((n, self.nq, 128), dtype=like.dtype, device=self.device), self.nq * 128
        rows, ld = self._rows(out, "out", self.nq, like.dtype)
        if rows != n:
            raise ValueError("out: one row for each row given is expected")
        return out, ld

    def append(self, qkv, seq, pos, rope, q_norm=None, k_norm=None, eps=1e-6, out=None):
        """Norms and turns the q and k heads of qkv [n, (nq + 2 nkv) * 128], stores keys and values at positions
        `pos` of sequences `seq` (int32 [n]; a position < 0 skips its row) and returns the queries [n, nq, 128].
        rope: float32 [rows, 64, 2], cosine and sine of each pair at each position."""
        from torch import float32, int32
        c = self._act(qkv)
        n, ld = self._rows(qkv, "qkv", self.nq + 2 * self.nkv)
        out, ldo = self._out(out, n, qkv)
        dev, rows = self._dev, rope.shape[0]
        _on_stream(dev, lambda stream: self._lib.q3paged_append(
            c, n, qkv.data_ptr(), ld, _need(seq, "seq", int32, (n,), dev), _need(pos, "pos", int32, (n,), dev),
            None if q_norm is None else _need(q_norm, "q_norm", float32, (128,), dev),
            None if k_norm is None else _need(k_norm, "k_norm", float32, (128,), dev), eps,
            _need(rope, "rope", float32, (rows, 64, 2), dev), rows, out.data_ptr(), ldo, self._err, stream))
        return out

    def attend(self, q, q_off, ctx_len, max_q: int, scale=128 ** -0.5, out=None):
        """Causal attention of the newest tokens of every sequence: rows q_off[s]..q_off[s+1]-1 of q [n, nq, 128]
        are the last ones of sequence s, which has ctx_len[s] positions (int32 tensors); max_q bounds the new
        tokens of a sequence.  Returns [n, nq, 128]; `out` may be q itself."""
        from torch import int32
        c = self._act(q)
        n, ld = self._rows(q, "q", self.nq)
        out, ldo = self._out(out, n, q)
        off = _need(q_off, "q_off", int32, self._q_off_shape, self._dev)
        ctx = _need(ctx_len, "ctx_len", int32, self._ctx_shape, self._dev)
        _on_stream(self._dev, lambda stream: self._lib.q3paged_attention(
            c, n, max_q, q.data_ptr(), ld, off, ctx, scale, out.data_ptr(), ldo, self._workspace(stream).data_ptr(),
            self.ws_bytes, self._err, stream))
        return out

    def check(self):
        """Waits for the device and raises where it met a page, position or length out of range since the last check."""
        import torch
        torch.cuda.synchronize(self.device)
        e = int(self.err.item())
        if e:
            self.err.zero_()
            raise Q3Error(Q3_ERR_TIMEOUT if e & Q3PAGED_ERR_TIMEOUT else Q3_ERR_BOUNDS,
                          "a device wait timed out" if e & Q3PAGED_ERR_TIMEOUT else
                          "a page, position or length is out of range")


def sample_given(logits, u, temperature, top_k, top_p, min_p, ids=None, logprob=None, err=None):
    """Draws one id for each row of logits ([n, vocab], float32 or bfloat16) from the given uniform numbers u,
    everything on the GPU and queued on the current stream: u, temperature, top_p, min_p float32 [n], top_k
    int32 [n].  Returns (ids int32 [n], log probabilities float32 [n]); an id is -1 where a row's logits hold
    NaN, +inf or nothing finite (q3tts_sample_given in q3tts.h has the definition)."""
    import torch
    if not (isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dim() == 2 and
            (logits.shape[1] <= 1 or logits.stride(1) == 1)):
        raise ValueError("logits: a CUDA tensor [n, vocab] with contiguous rows is expected")
    (n, vocab), dev, f = logits.shape, logits.get_device(), torch.float32
    if n > 1 and logits.stride(0) < vocab:
        raise ValueError("logits: rows must not share memory")
    if ids is None:
        ids = torch.empty(n, dtype=torch.int32, device=logits.device)
    if logprob is None:
        logprob = torch.empty(n, dtype=f, device=logits.device)
    shape = (n,)
    args = (_need(u, "u", f, shape, dev), _need(temperature, "temperature", f, shape, dev),
            _need(top_k, "top_k", torch.int32, shape, dev), _need(top_p, "top_p", f, shape, dev),
            _need(min_p, "min_p", f, shape, dev), _need(ids, "ids", torch.int32, shape, dev),
            _need(logprob, "logprob", f, shape, dev),
            None if err is None else _need(err, "err", torch.int32, (1,), dev))
    _on_stream(dev, lambda stream: lib().q3tts_sample_given(
        n, vocab, logits.data_ptr(), _dtype_code(logits), logits.stride(0) if n > 1 else vocab, *args, stream))
    return ids, logprob
