"""B200-native split residual vector quantiser of the Mimi codec (the tokenizer
bottleneck behind Moshi): encode 512-d latents to 8 codes per 80 ms frame
(1 semantic VQ + 7-level acoustic RVQ, 2048 codewords each) and decode them back.

This module is argument marshalling over the C ABI in ``include/mimi_rvq.h``
(``libmimi_rvq.so``, built by ``build.py``): every step of the computation runs
in the library's sm_100a kernels. PyTorch supplies device memory and streams
only. There is no fallback: if the library is missing or fails to load, using
this module raises.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import os

LATENT_DIM, DIM, CODEBOOK_SIZE, NUM_CODEBOOKS = 512, 256, 2048, 8
F32, BF16 = 0, 1
STATUS = {0: "ok", -1: "invalid argument", -2: "out of device memory", -3: "CUDA error",
          -4: "code out of range", -5: "device is not sm_100", -6: "kernel wait timed out"}

LIBRARY_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmimi_rvq.so")
EXPORTS = ("mimi_rvq_create", "mimi_rvq_destroy", "mimi_rvq_encode", "mimi_rvq_encode_ex",
           "mimi_rvq_encode_step", "mimi_rvq_project", "mimi_rvq_encode_scan", "mimi_rvq_decode",
           "mimi_rvq_decode_ex", "mimi_rvq_get_error", "mimi_rvq_stats", "mimi_rvq_strerror",
           "mimi_rvq_encode_profile", "mimi_rvq_delay_pack", "mimi_rvq_delay_unpack",
           "mimi_rvq_embed_sum", "mimi_rvq_wait_selftest", "mimi_rvq_encode_step_ex",
           "mimi_rvq_encode_noalloc", "mimi_rvq_streams_get_error",
           "mimi_rvq_streams_wait_selftest", "mimi_rvq_token_logprob",
           "mimi_rvq_token_logprob_grad", "mimi_rvq_distill_topk", "mimi_rvq_distill_topk_grad")
MAX_TOP, MAX_VOCAB, MAX_LOGIT_STREAMS = 128, 3 << 17, 65536
TEXT_CARD, TEXT_PAD, AUDIO_PAD = 32000, 32000, 2048

_lib = None


class MimiRVQError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, 'unknown')} (status {status})")
        self.status = status


def library() -> ctypes.CDLL:
    """Load libmimi_rvq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY_PATH):
        raise ImportError(f"{LIBRARY_PATH} is missing: build it with "
                          "`python -m split_residual_vector_b200.build`")
    lib = ctypes.CDLL(LIBRARY_PATH)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.mimi_rvq_create.argtypes = [vp, vp, vp, ctypes.POINTER(vp)]
    lib.mimi_rvq_create.restype = ci
    lib.mimi_rvq_destroy.argtypes = [vp]
    lib.mimi_rvq_destroy.restype = None
    lib.mimi_rvq_encode.argtypes = [vp, vp, ci, i64, vp, vp]
    lib.mimi_rvq_encode.restype = ci
    for name in ("mimi_rvq_encode_ex", "mimi_rvq_encode_scan"):
        getattr(lib, name).argtypes = [vp, vp, ci, i64, ci, ci, vp, vp]
        getattr(lib, name).restype = ci
    lib.mimi_rvq_encode_profile.argtypes = [vp, vp, ci, i64, vp, vp, vp]
    lib.mimi_rvq_encode_profile.restype = ci
    lib.mimi_rvq_project.argtypes = [vp, vp, ci, i64, vp, vp]
    lib.mimi_rvq_project.restype = ci
    lib.mimi_rvq_decode_ex.argtypes = [vp, vp, i64, ci, vp, vp]
    lib.mimi_rvq_decode_ex.restype = ci
    lib.mimi_rvq_encode_step.argtypes = [vp, vp, ci, ci, vp, vp]
    lib.mimi_rvq_encode_step.restype = ci
    lib.mimi_rvq_decode.argtypes = [vp, vp, i64, vp, vp]
    lib.mimi_rvq_decode.restype = ci
    lib.mimi_rvq_get_error.argtypes = [vp, vp]
    lib.mimi_rvq_get_error.restype = ci
    lib.mimi_rvq_stats.argtypes = [vp, vp, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.mimi_rvq_stats.restype = ci
    lib.mimi_rvq_strerror.argtypes = [ci]
    lib.mimi_rvq_strerror.restype = ctypes.c_char_p
    lib.mimi_rvq_encode_step_ex.argtypes = [vp, vp, ci, ci, ci, ci, vp, vp]
    lib.mimi_rvq_encode_step_ex.restype = ci
    lib.mimi_rvq_wait_selftest.argtypes = [vp, ci, vp]
    lib.mimi_rvq_wait_selftest.restype = ci
    lib.mimi_rvq_set_cluster_form.argtypes = [vp, ci]
    lib.mimi_rvq_set_cluster_form.restype = ci
    i32 = ctypes.c_int32
    lib.mimi_rvq_delay_pack.argtypes = [vp, vp, ci, i64, vp, i64, i32, i32, vp, vp]
    lib.mimi_rvq_delay_pack.restype = ci
    lib.mimi_rvq_delay_unpack.argtypes = [vp, i64, ci, ci, vp, i64, vp, vp]
    lib.mimi_rvq_delay_unpack.restype = ci
    lib.mimi_rvq_embed_sum.argtypes = [vp, ci, ci, vp, ci, vp, i64, vp, ci, vp, vp]
    lib.mimi_rvq_embed_sum.restype = ci
    lib.mimi_rvq_streams_get_error.argtypes = [vp]
    lib.mimi_rvq_streams_get_error.restype = ci
    lib.mimi_rvq_streams_wait_selftest.argtypes = [vp]
    lib.mimi_rvq_streams_wait_selftest.restype = ci
    rows = [vp, ci, i64, ci, ci, i64, i64]  # logits, dtype, S, n, V, strides
    toks = [vp, i64, i64, i32, ctypes.c_float]  # tokens, strides, pad, scale
    lib.mimi_rvq_token_logprob.argtypes = rows + toks + [ci] + [vp] * 7
    lib.mimi_rvq_token_logprob.restype = ci
    lib.mimi_rvq_token_logprob_grad.argtypes = rows + toks + [vp] * 4 + [i64] * 2 + [vp] * 5
    lib.mimi_rvq_token_logprob_grad.restype = ci
    teacher = [vp, vp, ci, ci, ci, ctypes.c_float]  # ids, teacher, dtype, k, tail, scale
    lib.mimi_rvq_distill_topk.argtypes = rows + teacher + [vp] * 3
    lib.mimi_rvq_distill_topk.restype = ci
    lib.mimi_rvq_distill_topk_grad.argtypes = rows + teacher + [vp] * 2 + [i64] * 2 + [vp] * 3
    lib.mimi_rvq_distill_topk_grad.restype = ci
    _lib = lib
    return lib


def strerror(status: int) -> str:
    return library().mimi_rvq_strerror(int(status)).decode()


def _check(status: int, what: str):
    if status != 0:
        raise MimiRVQError(status, what)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_flag(t):
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("latents must be float32 or bfloat16")


class Quantizer:
    """A library handle: codebooks [8, 2048, 256], W_in [256, 512], W_out [512, 256]
    (float32 CUDA tensors, copied at construction)."""

    def __init__(self, codebooks, W_in, W_out):
        import torch
        lib = library()
        cb = codebooks.detach().to(device="cuda", dtype=torch.float32).contiguous()
        wi = W_in.detach().to(device=cb.device, dtype=torch.float32).contiguous()
        wo = W_out.detach().to(device=cb.device, dtype=torch.float32).contiguous()
        assert cb.shape == (NUM_CODEBOOKS, CODEBOOK_SIZE, DIM), cb.shape
        assert wi.shape == (DIM, LATENT_DIM) and wo.shape == (LATENT_DIM, DIM)
        self.device = cb.device
        self._h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib.mimi_rvq_create(cb.data_ptr(), wi.data_ptr(), wo.data_ptr(),
                                       ctypes.byref(self._h)), "mimi_rvq_create")

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            library().mimi_rvq_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _codes_out(self, n, out, n_q=NUM_CODEBOOKS):
        import torch
        if out is None:
            out = torch.empty((n, n_q), dtype=torch.int16, device=self.device)
        assert out.dtype == torch.int16 and out.is_contiguous() and out.shape == (n, n_q)
        return out

    @staticmethod
    def _latents(latents):
        assert latents.dim() == 2 and latents.shape[1] == LATENT_DIM and latents.is_contiguous()
        return latents.shape[0], _dtype_flag(latents)

    def encode(self, latents, n_q=NUM_CODEBOOKS, variant=0, out=None, stream=None):
        """latents [N, 512] float32 / bfloat16 (CUDA) -> codes [N, n_q] int16."""
        n, dt = self._latents(latents)
        out = self._codes_out(n, out, n_q)
        if n_q == NUM_CODEBOOKS and variant == 0:
            st = library().mimi_rvq_encode(self._h, latents.data_ptr(), dt, n, out.data_ptr(),
                                           _stream(stream))
        else:
            st = library().mimi_rvq_encode_ex(self._h, latents.data_ptr(), dt, n, n_q, variant,
                                              out.data_ptr(), _stream(stream))
        _check(st, "mimi_rvq_encode")
        return out

    def encode_step(self, frames, out=None, stream=None, n_q=NUM_CODEBOOKS, variant=0):
        """frames [B, 512] (one frame per stream) -> codes [B, n_q] int16."""
        b, dt = self._latents(frames)
        out = self._codes_out(b, out, n_q)
        if n_q == NUM_CODEBOOKS and variant == 0:
            st = library().mimi_rvq_encode_step(self._h, frames.data_ptr(), dt, b, out.data_ptr(),
                                                _stream(stream))
        else:
            st = library().mimi_rvq_encode_step_ex(self._h, frames.data_ptr(), dt, b, n_q, variant,
                                                   out.data_ptr(), _stream(stream))
        _check(st, "mimi_rvq_encode_step")
        return out

    def project(self, latents, out=None, stream=None):
        """latents [N, 512] -> y = W_in z [N, 256] float32 (the encoder's projection step)."""
        import torch
        n, dt = self._latents(latents)
        if out is None:
            out = torch.empty((n, DIM), dtype=torch.float32, device=self.device)
        assert out.dtype == torch.float32 and out.is_contiguous() and out.shape == (n, DIM)
        _check(library().mimi_rvq_project(self._h, latents.data_ptr(), dt, n, out.data_ptr(),
                                          _stream(stream)), "mimi_rvq_project")
        return out

    def encode_scan(self, latents, n_q=NUM_CODEBOOKS, variant=0, out=None, stream=None):
        """Float32 full-scan encoder on CUDA cores (slow; for comparison)."""
        n, dt = self._latents(latents)
        out = self._codes_out(n, out, n_q)
        _check(library().mimi_rvq_encode_scan(self._h, latents.data_ptr(), dt, n, n_q, variant,
                                              out.data_ptr(), _stream(stream)),
               "mimi_rvq_encode_scan")
        return out

    def decode(self, codes, out=None, stream=None):
        """codes [N, n_q] int16 (CUDA) -> latents [N, 512] float32 (n_q = codes.shape[1])."""
        import torch
        assert codes.dtype == torch.int16 and codes.is_contiguous() and codes.dim() == 2
        n, n_q = codes.shape
        if out is None:
            out = torch.empty((n, LATENT_DIM), dtype=torch.float32, device=self.device)
        assert out.dtype == torch.float32 and out.is_contiguous() and out.shape == (n, LATENT_DIM)
        if n_q == NUM_CODEBOOKS:
            st = library().mimi_rvq_decode(self._h, codes.data_ptr(), n, out.data_ptr(),
                                           _stream(stream))
        else:
            st = library().mimi_rvq_decode_ex(self._h, codes.data_ptr(), n, n_q, out.data_ptr(),
                                              _stream(stream))
        _check(st, "mimi_rvq_decode")
        return out

    PROFILE_SLOTS = ("producer_wait_stage", "mma_wait_operands", "mma_wait_score_buffer",
                     "mma_wait_level_operand", "mma_wait_latents", "epi_wait_score_tile",
                     "epi_scan", "epi_pick", "epi_update", "epi_stage", "epi_barrier",
                     "cta_total", "n_chunks", "n_displaced", "n_runner_up", "n_more",
                     "pick_exchange_merge", "pick_rescore", "pick_select", "scan_drain",
                     "update_wait_operand", "update_work", "update_sync", "unused")
    PROFILE_COUNTS = ("n_chunks", "n_displaced", "n_runner_up", "n_more")

    def encode_profile(self, latents, out=None, stream=None):
        """Encode and return (codes, {role: cycles summed over CTAs}) from the kernel's
        self-profile; the PROFILE_COUNTS entries are event counts, not cycles."""
        import torch
        n, dt = self._latents(latents)
        out = self._codes_out(n, out)
        cyc = torch.zeros(len(self.PROFILE_SLOTS), dtype=torch.int64, device=self.device)
        _check(library().mimi_rvq_encode_profile(self._h, latents.data_ptr(), dt, n,
                                                 out.data_ptr(), cyc.data_ptr(), _stream(stream)),
               "mimi_rvq_encode_profile")
        vals = cyc.cpu().tolist()
        return out, dict(zip(self.PROFILE_SLOTS, vals))

    def wait_selftest(self, which: int, stream=None):
        """Launch a kernel whose wait never completes (0: mbarrier, 1: group barrier); it
        times out after ~50 ms. The next get_error() returns -6 (timed out)."""
        _check(library().mimi_rvq_wait_selftest(self._h, int(which), _stream(stream)),
               "mimi_rvq_wait_selftest")

    def set_cluster_form(self, enabled: bool):
        """Use the thread-block-cluster form of the float32 latency encoder (default where the
        device runs clusters) or the group form, for streaming steps of up to 256 frames and
        the float32 re-encode after a batch encode."""
        _check(library().mimi_rvq_set_cluster_form(self._h, 1 if enabled else 0),
               "mimi_rvq_set_cluster_form")

    def get_error(self, stream=None) -> int:
        """Synchronise the stream; return and clear the device error status (0 = ok)."""
        return int(library().mimi_rvq_get_error(self._h, _stream(stream)))

    def stats(self, stream=None):
        """(frames encoded, frames whose candidates could not be certified and were resolved in
        float32: re-encoded after a batch encode, scanned exactly in a sliced step) since create."""
        a, b = ctypes.c_int64(), ctypes.c_int64()
        _check(library().mimi_rvq_stats(self._h, _stream(stream), ctypes.byref(a),
                                        ctypes.byref(b)), "mimi_rvq_stats")
        return a.value, b.value


# ----------------------------------------------------------------- token streams


def _host_i32(values, n):
    arr = (ctypes.c_int32 * n)(*[int(v) for v in values])
    assert len(values) == n
    return arr


def delay_pack(text, audio, delays, S=None, text_pad=TEXT_PAD, audio_pad=AUDIO_PAD, out=None,
               stream=None):
    """Multi-stream sequence [S, 1 + 8 * n_audio] int32 from text [T] int32 (or None) and
    audio codes [n_audio, T, 8] int16 (CUDA), level q shifted later by delays[q] steps.
    S defaults to T + max(delays)."""
    import torch
    assert audio.dtype == torch.int16 and audio.dim() == 3 and audio.shape[2] == NUM_CODEBOOKS
    assert audio.is_contiguous()
    n_audio, T, _ = audio.shape
    S = T + max(int(v) for v in delays) if S is None else int(S)
    K = 1 + NUM_CODEBOOKS * n_audio
    if text is not None:
        assert text.dtype == torch.int32 and text.is_contiguous() and text.shape == (T,)
    if out is None:
        out = torch.empty((S, K), dtype=torch.int32, device=audio.device)
    assert out.dtype == torch.int32 and out.is_contiguous() and out.shape == (S, K)
    _check(library().mimi_rvq_delay_pack(None if text is None else text.data_ptr(),
                                         audio.data_ptr(), n_audio, T,
                                         _host_i32(delays, NUM_CODEBOOKS), S, int(text_pad),
                                         int(audio_pad), out.data_ptr(), _stream(stream)),
           "mimi_rvq_delay_pack")
    return out


def delay_unpack(packed, col0, delays, T=None, out=None, stream=None):
    """Audio codes [T, 8] int16 from the 8 columns of packed [S, K] int32 that start at col0
    (the inverse shift). T defaults to S - max(delays)."""
    import torch
    assert packed.dtype == torch.int32 and packed.dim() == 2 and packed.is_contiguous()
    S, K = packed.shape
    T = S - max(int(v) for v in delays) if T is None else int(T)
    if out is None:
        out = torch.empty((T, NUM_CODEBOOKS), dtype=torch.int16, device=packed.device)
    assert out.dtype == torch.int16 and out.is_contiguous() and out.shape == (T, NUM_CODEBOOKS)
    _check(library().mimi_rvq_delay_unpack(packed.data_ptr(), S, K, int(col0),
                                           _host_i32(delays, NUM_CODEBOOKS), T, out.data_ptr(),
                                           _stream(stream)), "mimi_rvq_delay_unpack")
    return out


def embed_sum(tables, rows, tokens, out_dtype=None, out=None, n_bad=None, stream=None):
    """out [S, d] = sum over k of row tokens[s, k] of table k. tables: stacked rows
    [sum(rows), d] float32 / bfloat16 (CUDA); rows: the K row counts; tokens [S, K] int32.
    n_bad: optional CUDA int64 [1] (caller-zeroed) counting tokens past their table."""
    import torch
    assert tables.dim() == 2 and tables.is_contiguous()
    assert tokens.dtype == torch.int32 and tokens.dim() == 2 and tokens.is_contiguous()
    S, K = tokens.shape
    d = tables.shape[1]
    assert len(rows) == K and sum(int(r) for r in rows) == tables.shape[0]
    if out is None:
        out = torch.empty((S, d), dtype=out_dtype or tables.dtype, device=tables.device)
    assert out.is_contiguous() and out.shape == (S, d)
    host_rows = (ctypes.c_int64 * K)(*[int(r) for r in rows])
    _check(library().mimi_rvq_embed_sum(tables.data_ptr(), _dtype_flag(tables), K, host_rows, d,
                                        tokens.data_ptr(), S, out.data_ptr(), _dtype_flag(out),
                                        None if n_bad is None else n_bad.data_ptr(),
                                        _stream(stream)), "mimi_rvq_embed_sum")
    return out


def streams_get_error(stream=None) -> int:
    """Synchronise the stream; return and clear the token-stream status word (0 = ok, -6 =
    a wait of embed_sum timed out)."""
    return int(library().mimi_rvq_streams_get_error(_stream(stream)))


def streams_wait_selftest(stream=None):
    """Launch the embedding-sum kernel in its self-test form: its wait never completes and
    times out after ~50 ms; the next streams_get_error() returns -6."""
    _check(library().mimi_rvq_streams_wait_selftest(_stream(stream)),
           "mimi_rvq_streams_wait_selftest")


# ----------------------------------------------------------------- logits over the streams

TokenLogprobs = collections.namedtuple("TokenLogprobs",
                                       "logprob entropy lse top_ids top_logprob")
TokenLogprobs.__doc__ = """Values of token_logprobs: logprob, entropy, lse [S(, n)] float32,
top_ids [S(, n), k] int32 and top_logprob [S(, n), k] float32; None where not wanted."""


@contextlib.contextmanager
def _current(device, stream):
    """`device` and `stream` (None: the device's current stream) made current, so that outputs
    are allocated there too."""
    import torch
    if stream is None:
        with torch.cuda.device(device):
            yield
    else:
        assert stream.device == device, "the stream belongs to another device than the logits"
        with torch.cuda.stream(stream), torch.cuda.device(device):
            yield


def _elsewhere(device, stream):
    """Whether a call has to make its device or stream current first."""
    import torch
    return stream is not None or device.index != torch.cuda.current_device()


def _raw_stream(device):
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _list_length(k, what):
    """k, refused here where the C argument would not hold it (or an output would be large)."""
    if not 0 <= k <= MAX_TOP:
        raise MimiRVQError(-1, what)
    return k


def _new_values(lead, device, tokens, top_k):
    """Outputs of token_logprobs and their pointers."""
    import torch
    entropy = torch.empty(*lead, dtype=torch.float32, device=device)
    lse = torch.empty_like(entropy)
    logprob = ids = top = p_logprob = p_ids = p_top = None
    if tokens is not None:
        logprob = torch.empty_like(entropy)
        p_logprob = logprob.data_ptr()
    if top_k:
        top = torch.empty(*lead, top_k, dtype=torch.float32, device=device)
        ids = torch.empty_like(top, dtype=torch.int32)
        p_ids, p_top = ids.data_ptr(), top.data_ptr()
    return (TokenLogprobs(logprob, entropy, lse, ids, top),
            (p_logprob, entropy.data_ptr(), lse.data_ptr(), p_ids, p_top))


def _given_values(v, lead, device, top_k):
    """The same of outputs that the caller gave."""
    import torch
    f32, top = torch.float32, (*lead, top_k)
    return v, (_row_array(v.logprob, lead, f32, device), _row_array(v.entropy, lead, f32, device),
               _row_array(v.lse, lead, f32, device), _row_array(v.top_ids, top, torch.int32, device),
               _row_array(v.top_logprob, top, f32, device))


def _logit_rows(logits):
    """(lead shape, dtype flag, S, n, V, stride_s, stride_n) of [S, V] or [S, n, V] logits."""
    shape, stride = logits.shape, logits.stride()
    dims, V = len(shape), shape[-1]
    assert logits.is_cuda and dims in (2, 3), "logits are [S, V] or [S, n, V] on CUDA"
    assert V <= 1 or stride[-1] == 1, "a row's logits are contiguous"
    assert V <= MAX_VOCAB, f"rows have at most {MAX_VOCAB} logits"
    assert dims == 2 or shape[1] <= MAX_LOGIT_STREAMS, f"at most {MAX_LOGIT_STREAMS} streams"
    if dims == 2:
        return shape[:1], _dtype_flag(logits), shape[0], 1, V, stride[0], 0
    return shape[:2], _dtype_flag(logits), shape[0], shape[1], V, stride[0], stride[1]


def _row_tokens(tokens, pad, lead, device):
    """(pointer, stride_s, stride_n, pad) of tokens of the rows' shape, any strides."""
    import torch
    assert -(1 << 31) <= pad < 1 << 31, "pad is an int32"
    if tokens is None:
        return None, 0, 0, pad
    assert tokens.dtype == torch.int32 and tokens.shape == lead and tokens.device == device
    st = tokens.stride()
    return tokens.data_ptr(), st[0], st[1] if len(st) == 2 else 0, pad


def _row_array(t, shape, dtype, device):
    """Pointer of a contiguous array of that shape, None for None."""
    if t is None:
        return None
    assert t.dtype == dtype and t.shape == shape and t.is_contiguous() and t.device == device
    return t.data_ptr()


def _bad_counter(n_bad, device):
    if n_bad is None:
        return None
    import torch
    assert n_bad.dtype == torch.int64 and n_bad.numel() >= 1 and n_bad.device == device
    return n_bad.data_ptr()


def _gradient(out, logits):
    """The gradient's tensor and its (stride_s, stride_n). A new one is contiguous, or stream-major
    where the logits are (its rows are then aligned as theirs, and stored as whole vectors)."""
    import torch
    if out is None:
        shape = logits.shape
        if len(shape) == 3 and logits.stride() == (shape[2], shape[0] * shape[2], 1):
            out = torch.empty_like(logits)
        else:
            out = torch.empty(*shape, dtype=logits.dtype, device=logits.device)
    assert out.shape == logits.shape and out.dtype == logits.dtype and out.device == logits.device
    st = out.stride()
    assert out.shape[-1] <= 1 or st[-1] == 1
    return out, (st[0], st[1] if out.dim() == 3 else 0)


def token_logprobs(logits, tokens=None, pad=-1, scale=1.0, top_k=0, out=None, n_bad=None,
                   stream=None):
    """Log probabilities of the streams' tokens: logits [S, V] or [S, n, V] float32 / bfloat16
    (CUDA, rows contiguous, any strides between rows), tokens [S] or [S, n] int32 (a view such
    as packed[:, 1:9] is read in place; below 0 or equal to pad: no target, logprob 0).
    Returns TokenLogprobs; logprob is None without tokens, the top lists are None for
    top_k = 0. scale is 1 / temperature (1e-30 to 1e30). out: TokenLogprobs of tensors to
    write, None in the place of values that are not wanted. n_bad: optional CUDA int64 [1]
    (caller-zeroed) counting tokens past V."""
    lead, dt, S, n, V, ss, sn = _logit_rows(logits)
    dev, top_k = logits.device, _list_length(int(top_k), "mimi_rvq_token_logprob")
    if _elsewhere(dev, stream):
        with _current(dev, stream):
            return token_logprobs(logits, tokens, pad, scale, top_k, out, n_bad)
    v, pointers = (_new_values(lead, dev, tokens, top_k) if out is None
                   else _given_values(out, lead, dev, top_k))
    _check(library().mimi_rvq_token_logprob(
        logits.data_ptr(), dt, S, n, V, ss, sn, *_row_tokens(tokens, pad, lead, dev), scale,
        top_k, *pointers, _bad_counter(n_bad, dev), _raw_stream(dev)), "mimi_rvq_token_logprob")
    return v


def token_logprobs_grad(logits, tokens=None, g_logprob=None, g_entropy=None, g_lse=None, pad=-1,
                        scale=1.0, values=None, out=None, n_bad=None, stream=None):
    """Gradient of sum(g_logprob * logprob + g_entropy * entropy + g_lse * lse) with respect to
    the logits, in the logits' type: g_* are [S] or [S, n] float32, None where there is none.
    out may be the logits themselves; a new gradient is contiguous, or stream-major where the
    logits are dense and stream-major. values = True, or a TokenLogprobs of tensors (top lists
    None), also gives logprob, entropy and lse from the same pass: the call then returns
    (dlogits, TokenLogprobs). Otherwise it returns dlogits."""
    import torch
    lead, dt, S, n, V, ss, sn = _logit_rows(logits)
    dev, f32 = logits.device, torch.float32
    if _elsewhere(dev, stream):
        with _current(dev, stream):
            return token_logprobs_grad(logits, tokens, g_logprob, g_entropy, g_lse, pad, scale,
                                       values, out, n_bad)
    d, d_strides = _gradient(out, logits)
    if not values:
        v, pointers = None, (None, None, None)
    else:
        v, pointers = (_new_values(lead, dev, tokens, 0) if values is True
                       else _given_values(values, lead, dev, 0))
        assert v.top_ids is None and v.top_logprob is None, "the gradient call lists no tokens"
    _check(library().mimi_rvq_token_logprob_grad(
        logits.data_ptr(), dt, S, n, V, ss, sn, *_row_tokens(tokens, pad, lead, dev), scale,
        _row_array(g_logprob, lead, f32, dev), _row_array(g_entropy, lead, f32, dev),
        _row_array(g_lse, lead, f32, dev), d.data_ptr(), *d_strides, *pointers[:3],
        _bad_counter(n_bad, dev), _raw_stream(dev)), "mimi_rvq_token_logprob_grad")
    return (d, v) if values else d


def _teacher_list(ids, teacher, lead, device):
    """(ids, teacher, teacher dtype, k) of a teacher's lists [S(, n), k]."""
    import torch
    assert ids.dim() == len(lead) + 1 and teacher.dtype in (torch.float32, torch.bfloat16)
    shape = (*lead, _list_length(ids.shape[-1], "mimi_rvq_distill_topk"))
    return (_row_array(ids, shape, torch.int32, device),
            _row_array(teacher, shape, teacher.dtype, device), _dtype_flag(teacher), shape[-1])


def distill_topk(logits, ids, teacher, tail=False, scale=1.0, out=None, n_bad=None, stream=None):
    """Loss [S] or [S, n] float32 of a student's logits against a teacher's top lists: ids
    [S(, n), k] int32 (below 0: empty) and teacher [S(, n), k] float32 / bfloat16 as
    token_logprobs(..., top_k=k) gives them. tail = False: KL to the list's softmax; tail =
    True: the teacher's log probabilities as they are, with all other tokens as one more
    class. scale applies to the student only."""
    import torch
    lead, dt, S, n, V, ss, sn = _logit_rows(logits)
    dev, f32 = logits.device, torch.float32
    if _elsewhere(dev, stream):
        with _current(dev, stream):
            return distill_topk(logits, ids, teacher, tail, scale, out, n_bad)
    loss = torch.empty(*lead, dtype=f32, device=dev) if out is None else out
    _check(library().mimi_rvq_distill_topk(
        logits.data_ptr(), dt, S, n, V, ss, sn, *_teacher_list(ids, teacher, lead, dev),
        1 if tail else 0, scale, _row_array(loss, lead, f32, dev), _bad_counter(n_bad, dev),
        _raw_stream(dev)), "mimi_rvq_distill_topk")
    return loss


def distill_topk_grad(logits, ids, teacher, g=None, tail=False, scale=1.0, loss=None, out=None,
                      n_bad=None, stream=None):
    """Gradient of sum(g * loss) with respect to the logits, in their type (g [S] or [S, n]
    float32, None: all 1; out may be the logits themselves, a new gradient is laid out as
    token_logprobs_grad's). loss = True, or a float32 tensor [S] or [S, n], also gives the
    losses from the same pass: the call then returns (dlogits, loss). Otherwise (None, False)
    it returns dlogits."""
    import torch
    lead, dt, S, n, V, ss, sn = _logit_rows(logits)
    dev, f32 = logits.device, torch.float32
    if _elsewhere(dev, stream):
        with _current(dev, stream):
            return distill_topk_grad(logits, ids, teacher, g, tail, scale, loss, out, n_bad)
    d, d_strides = _gradient(out, logits)
    if loss is True:
        loss = torch.empty(*lead, dtype=f32, device=dev)
    elif loss is False:
        loss = None
    _check(library().mimi_rvq_distill_topk_grad(
        logits.data_ptr(), dt, S, n, V, ss, sn, *_teacher_list(ids, teacher, lead, dev),
        1 if tail else 0, scale, _row_array(g, lead, f32, dev), d.data_ptr(), *d_strides,
        _row_array(loss, lead, f32, dev), _bad_counter(n_bad, dev), _raw_stream(dev)),
        "mimi_rvq_distill_topk_grad")
    return d if loss is None else (d, loss)
