"""ctypes binding of the scoring-head operators (include/rbf_ops.h), argument
marshalling only: 8-bit row quantisation, the 8-bit integer product with a
scale for each token and channel, a linear layer on 8-bit weights, sampling from
scores, 8-bit floating-point rows and their product with a scale for each block
of 128, verification of drafted tokens, and distillation from a teacher's best
logits. All of it runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes

from . import _binding
from ._binding import RBF_OK, RbfError, load_library

RBF_DTYPE_F32 = 0
RBF_DTYPE_BF16 = 1
RBF_DTYPE_F16 = 2
RBF_DTYPE_I32 = 3
RBF_DTYPE_E4M3 = 5
RBF_DTYPE_E5M2 = 6
RBF_OPS_MAX_DEPTH = 65536
RBF_OPS_MAX_VOCAB = 1 << 26
RBF_OPS_MAX_DRAFTS = 1024
RBF_OPS_MAX_TEACHER = 1024

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_S = ctypes.c_int
_F = ctypes.c_float
_binding.SIGNATURES.update({
    "rbf_ops_create": (_S, [_I64, _I32, _P, ctypes.POINTER(_P)]),
    "rbf_ops_destroy": (_S, [_P]),
    "rbf_ops_device": (_I32, [_P]),
    "rbf_ops_stream": (_P, [_P]),
    "rbf_ops_last_cuda_error": (_I32, [_P]),
    "rbf_ops_last_launches": (_I32, [_P]),
    "rbf_ops_check_device_error": (_S, [_P]),
    "rbf_ops_set_timeout": (_S, [_P, _I64]),
    "rbf_ops_inject_host_fault": (_S, [_P, _I32]),
    "quantize_rows_i8_dev": (_S, [_P, _P, _S, _I64, _I64, _I32, _P, _I64, _P]),
    "matmul_i8_dev": (_S, [_P, _P, _I64, _P, _P, _I64, _P, _P, _P, _S, _I64, _I64, _I64, _I32]),
    "linear_i8_dev": (_S, [_P, _P, _S, _I64, _P, _I64, _P, _P, _P, _S, _I64, _I64, _I64, _I32]),
    "sample_dev": (_S, [_P, _P, _S, _I64, _I64, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "quantize_f8_dev": (_S, [_P, _P, _S, _I64, _I64, _I32, _I32, _P, _S, _I64, _P, _I64]),
    "matmul_f8_dev": (_S, [_P, _P, _S, _I64, _P, _I64, _P, _S, _I64, _P, _I64, _I32, _P, _P, _S, _I64, _I64, _I64, _I32]),
    "verify_dev": (_S, [_P, _P, _I64, _I64, _P, _I64, _I64, _S, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "distill_dev": (_S, [_P, _P, _S, _I64, _I64, _I32, _P, _I64, _P, _S, _I64, _I32, _P, _P, _F, _P, _P, _I64]),
})

_STREAM_LEGACY = 1  # cudaStreamLegacy: the default stream, named explicitly
_DTYPES: dict = {}
_F8: dict = {}


def _dtypes() -> dict:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: RBF_DTYPE_F32, torch.bfloat16: RBF_DTYPE_BF16, torch.float16: RBF_DTYPE_F16,
                        torch.int32: RBF_DTYPE_I32, torch.int8: -1})
        _F8.update({torch.float8_e4m3fn: RBF_DTYPE_E4M3, torch.float8_e5m2: RBF_DTYPE_E5M2})
    return _DTYPES


# The checks below run before every launch: messages are put together only when one fails. Every call's first one
# is of a matrix' type, which fills _DTYPES.
# device: the handle's, which every tensor has to be on.

def _float_matrix(t, what: str, device, integers: bool = False):
    """Device pointer, row stride, rows, columns and dtype code of a 2-D CUDA tensor with contiguous rows."""
    code = _dtypes().get(t.dtype)
    if code is None or code < 0 or (code == RBF_DTYPE_I32 and not integers):
        raise TypeError(f"{what} is {t.dtype}: expected float32, bfloat16 or float16" + (" or int32" if integers else ""))
    return *_matrix(t, what, device), code


def _i8_matrix(t, what: str, device):
    if _dtypes().get(t.dtype) != -1:
        raise TypeError(f"{what} is {t.dtype}: expected int8")
    return _matrix(t, what, device)


def _f8_matrix(t, what: str, device):
    _dtypes()
    code = _F8.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} is {t.dtype}: expected float8_e4m3fn or float8_e5m2")
    return *_matrix(t, what, device), code


def _f32_matrix(t, rows: int, cols: int, what: str, device):
    """Device pointer and row stride of a float32 matrix of that shape."""
    if _dtypes().get(t.dtype) != RBF_DTYPE_F32:
        raise TypeError(f"{what} is {t.dtype}: expected float32")
    p, ld, got_rows, got_cols = _matrix(t, what, device)
    if (got_rows, got_cols) != (rows, cols):
        raise ValueError(f"the shape of {what} is {(got_rows, got_cols)}, expected {(rows, cols)}")
    return p, ld


def _places(t, seqs: int, places: int, what: str, device):
    """Device pointer, strides of a sequence and of a place, and dtype code of scores [seqs, places, vocab]."""
    code = _dtypes().get(t.dtype)
    if code is None or code < 0 or code == RBF_DTYPE_I32:
        raise TypeError(f"{what} is {t.dtype}: expected float32, bfloat16 or float16")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{what} is a 3-D tensor")
    if t.get_device() != device:
        _wrong_device(t, what, device)
    if (shape[0], shape[1]) != (seqs, places):
        raise ValueError(f"{what} has {shape[0]} sequences of {shape[1]} places, expected {seqs} of {places}")
    vocab = shape[2]
    if vocab > _INT32_MAX:
        raise ValueError(f"the rows of {what} have {vocab} values, more than 2^31 - 1")
    ld_seq, ld, step = t.stride()
    if vocab > 1 and step != 1:
        raise ValueError(f"{what}: the values of a row must be contiguous")
    if places <= 1:
        ld = max(ld, vocab, 1)  # one place: any stride
    elif ld < vocab:
        raise ValueError(f"{what}: rows overlap")
    room = (places - 1) * ld + vocab if places else 0
    if seqs <= 1:
        ld_seq = max(ld_seq, room, 1)
    elif ld_seq < room:
        raise ValueError(f"{what}: sequences overlap")
    return t.data_ptr(), ld_seq, ld, vocab, code


def _block_rows(scale_rows: int, rows: int) -> int:
    """1 or 128: how many rows share a scale, by the number of rows of scales."""
    return 1 if scale_rows == rows else 128


def _wrong_device(t, what: str, device) -> None:
    if not t.is_cuda:
        raise TypeError(f"{what}: expected a CUDA tensor")
    if device is not None:
        raise ValueError(f"{what} is on device {t.get_device()}, the handle on device {device}")


_INT32_MAX = 2 ** 31 - 1


def _matrix(t, what: str, device):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} is a 2-D tensor")
    if t.get_device() != device:
        _wrong_device(t, what, device)
    rows, cols = shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what}: the values of a row must be contiguous")
    if cols > _INT32_MAX:  # the library's type: ctypes would cut it to its low 32 bits
        raise ValueError(f"the rows of {what} have {cols} values, more than 2^31 - 1")
    if rows <= 1:
        ld = max(ld, cols, 1)  # one row: any stride
    elif ld < cols:
        raise ValueError(f"{what}: rows overlap")
    return t.data_ptr(), ld, rows, cols


def _int(value: int, bits: int) -> int:
    """A number as a signed integer of that many bits, at its limit where it is past that (the library refuses it)."""
    return max(-(1 << bits - 1), min(int(value), (1 << bits - 1) - 1))


def _vector(t, count: int, what: str, device, code: int = RBF_DTYPE_F32, optional: bool = True):
    if t is None:
        if not optional:
            raise ValueError(f"{what} is required")
        return None
    if t.numel() != count:
        raise ValueError(f"{what} has {t.numel()} entries, expected {count}")
    if t.get_device() != device:
        _wrong_device(t, what, device)
    if _DTYPES.get(t.dtype) != code:
        raise TypeError(f"{what} is {t.dtype}: expected {'int32' if code == RBF_DTYPE_I32 else 'float32'}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _same(got, want, what: str) -> None:
    if got != want:
        raise ValueError(f"{what} is {got}, expected {want}")


class Ops:
    """A handle with its stream and workspace (``rbf_ops_create``): products of
    up to ``max_rows`` rows of up to ``max_depth`` values (8-bit floating-point ones
    of any). Like an engine, one
    handle serves one call at a time; every call is enqueued on the handle's
    stream (``stream``: a torch stream or a raw handle; None: a stream of its
    own). The handle belongs to the device that was current then: tensors are on
    that one, and calls are made with it current. Outputs are given by the
    caller; a tensor used here must not be handed to another stream before this
    one has reached the call."""

    _device = None  # of the handle

    def __init__(self, max_rows: int, max_depth: int, stream=None):
        self.lib = load_library()
        s = None
        if stream is not None:
            s = (stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)) or _STREAM_LEGACY
        handle = ctypes.c_void_p()
        st = self.lib.rbf_ops_create(_int(max_rows, 64), _int(max_depth, 32), ctypes.c_void_p(s) if s else None,
                                     ctypes.byref(handle))
        if st != RBF_OK:
            raise RbfError(st, "rbf_ops_create")
        self._h = handle
        self._device = self.lib.rbf_ops_device(handle)
        self._stream_ref = stream

    # -- lifetime
    def close(self) -> None:
        if getattr(self, "_h", None):
            self.lib.rbf_ops_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _check(self, st: int, where: str) -> None:
        if st != RBF_OK:
            raise RbfError(st, where, self.lib.rbf_ops_last_cuda_error(self._h))

    # -- info
    @property
    def stream_handle(self) -> int:
        return self.lib.rbf_ops_stream(self._h) or 0

    @property
    def last_launches(self) -> int:
        """Kernels the most recent call enqueued."""
        return self.lib.rbf_ops_last_launches(self._h)

    def check_device_error(self) -> int:
        """Wait for the stream; the status its kernels reported since the last check."""
        return self.lib.rbf_ops_check_device_error(self._h)

    def set_timeout(self, nanoseconds: int) -> None:
        """Bound each device-side wait of later calls (default 2e9, at least 1e6); it does not limit a call's time."""
        self._check(self.lib.rbf_ops_set_timeout(self._h, _int(nanoseconds, 64)), "rbf_ops_set_timeout")

    def inject_host_fault(self, count: int) -> None:
        self._check(self.lib.rbf_ops_inject_host_fault(self._h, _int(count, 32)), "rbf_ops_inject_host_fault")

    # -- operators
    def quantize_rows_i8_dev(self, d_x, d_q, d_scale) -> None:
        """Rows of d_x [rows, cols] (float32, bfloat16 or float16) to int8 d_q with one scale a row in d_scale."""
        on = self._device
        x, ld_x, rows, cols, dtype = _float_matrix(d_x, "d_x", on)
        q, ld_q, q_rows, q_cols = _i8_matrix(d_q, "d_q", on)
        _same((q_rows, q_cols), (rows, cols), "the shape of d_q")
        self._check(self.lib.quantize_rows_i8_dev(self._h, x, dtype, ld_x, rows, cols, q, ld_q,
                                                  _vector(d_scale, rows, "d_scale", on, optional=False)),
                    "quantize_rows_i8_dev")

    def matmul_i8_dev(self, d_a, d_a_scale, d_b, d_b_scale, d_out, bias=None) -> None:
        """d_out [m, n] = d_a [m, k] times d_b [n, k] transposed, both int8, each row of either with its scale (None:
        1), plus bias [n]. An int32 d_out takes the sums themselves, without scales or bias."""
        on = self._device
        a, ld_a, m, k = _i8_matrix(d_a, "d_a", on)
        b, ld_b, n, b_cols = _i8_matrix(d_b, "d_b", on)
        out, ld_out, out_rows, out_cols, dtype = _float_matrix(d_out, "d_out", on, integers=True)
        _same(b_cols, k, "the depth of d_b")
        _same((out_rows, out_cols), (m, n), "the shape of d_out")
        self._check(self.lib.matmul_i8_dev(self._h, a, ld_a, _vector(d_a_scale, m, "d_a_scale", on), b, ld_b,
                                           _vector(d_b_scale, n, "d_b_scale", on), _vector(bias, n, "bias", on), out,
                                           dtype, ld_out, m, n, k), "matmul_i8_dev")

    def linear_i8_dev(self, d_x, d_w, d_w_scale, d_out, bias=None) -> None:
        """d_out [m, n] = d_x [m, k] (quantised by rows) times the int8 weights d_w [n, k] transposed, times the
        weights' row scales d_w_scale (None: 1), plus bias [n]."""
        on = self._device
        x, ld_x, m, k, x_dtype = _float_matrix(d_x, "d_x", on)
        w, ld_w, n, w_cols = _i8_matrix(d_w, "d_w", on)
        out, ld_out, out_rows, out_cols, dtype = _float_matrix(d_out, "d_out", on)
        _same(w_cols, k, "the depth of d_w")
        _same((out_rows, out_cols), (m, n), "the shape of d_out")
        self._check(self.lib.linear_i8_dev(self._h, x, x_dtype, ld_x, w, ld_w,
                                           _vector(d_w_scale, n, "d_w_scale", on), _vector(bias, n, "bias", on), out,
                                           dtype, ld_out, m, n, k), "linear_i8_dev")

    def sample_dev(self, d_logits, d_u, d_token, d_logprob=None, temperature=None, top_k=None, top_p=None,
                   min_p=None) -> None:
        """One index a row of d_logits [rows, vocab] into d_token (int32; -1 where every score is -infinity), and the
        log of its share into d_logprob. d_u: one random number in [0, 1) a row; temperature, top_p and min_p (float32)
        and top_k (int32): one entry a row, or None."""
        on = self._device
        x, ld, rows, vocab, dtype = _float_matrix(d_logits, "d_logits", on)
        self._check(self.lib.sample_dev(self._h, x, dtype, ld, rows, vocab,
                                        _vector(d_u, rows, "d_u", on, optional=False),
                                        _vector(temperature, rows, "temperature", on),
                                        _vector(top_k, rows, "top_k", on, RBF_DTYPE_I32),
                                        _vector(top_p, rows, "top_p", on),
                                        _vector(min_p, rows, "min_p", on),
                                        _vector(d_token, rows, "d_token", on, RBF_DTYPE_I32, optional=False),
                                        _vector(d_logprob, rows, "d_logprob", on)), "sample_dev")

    def quantize_f8_dev(self, d_x, d_q, d_scale, block_rows: int = 1) -> None:
        """d_x [rows, cols] (float32, bfloat16 or float16) to 8-bit floating point d_q (float8_e4m3fn or float8_e5m2),
        with one float32 scale for each 128 values of block_rows rows (1, or 128) in d_scale
        [ceil(rows / block_rows), ceil(cols / 128)]."""
        on = self._device
        x, ld_x, rows, cols, dtype = _float_matrix(d_x, "d_x", on)
        q, ld_q, q_rows, q_cols, q_dtype = _f8_matrix(d_q, "d_q", on)
        _same((q_rows, q_cols), (rows, cols), "the shape of d_q")
        if block_rows not in (1, 128):
            raise ValueError(f"block_rows is {block_rows}, expected 1 or 128")
        scale, ld_scale = _f32_matrix(d_scale, -(-rows // block_rows), -(-cols // 128), "d_scale", on)
        self._check(self.lib.quantize_f8_dev(self._h, x, dtype, ld_x, rows, cols, block_rows, q, q_dtype, ld_q, scale,
                                             ld_scale), "quantize_f8_dev")

    def matmul_f8_dev(self, d_a, d_a_scale, d_b, d_b_scale, d_out, bias=None) -> None:
        """d_out [m, n] = d_a [m, k] times d_b [n, k] transposed, both 8-bit floating point (either type), plus bias
        [n]. Each 128 values of a row of d_a have a scale, in d_a_scale [m, ceil(k / 128)], and so have those of d_b in
        d_b_scale [n, ceil(k / 128)], or those of 128 rows of it in d_b_scale [ceil(n / 128), ceil(k / 128)]. k may pass
        the handle's max_depth (up to RBF_OPS_MAX_VOCAB) where the rows start on 16-byte boundaries."""
        on = self._device
        a, ld_a, m, k, a_dtype = _f8_matrix(d_a, "d_a", on)
        b, ld_b, n, b_cols, b_dtype = _f8_matrix(d_b, "d_b", on)
        out, ld_out, out_rows, out_cols, dtype = _float_matrix(d_out, "d_out", on)
        _same(b_cols, k, "the depth of d_b")
        _same((out_rows, out_cols), (m, n), "the shape of d_out")
        blocks = -(-k // 128)
        a_scale, ld_a_scale = _f32_matrix(d_a_scale, m, blocks, "d_a_scale", on)
        block_rows = _block_rows(d_b_scale.shape[0], n)
        b_scale, ld_b_scale = _f32_matrix(d_b_scale, n if block_rows == 1 else -(-n // 128), blocks, "d_b_scale", on)
        self._check(self.lib.matmul_f8_dev(self._h, a, a_dtype, ld_a, a_scale, ld_a_scale, b, b_dtype, ld_b, b_scale,
                                           ld_b_scale, block_rows, _vector(bias, n, "bias", on), out, dtype, ld_out, m,
                                           n, k), "matmul_f8_dev")

    def verify_dev(self, d_target, d_draft_token, d_u, d_token, d_accepted, d_logprob=None, d_draft=None,
                   draft_count=None, temperature=None) -> None:
        """Drafted tokens d_draft_token [seqs, drafts] (int32) checked against the target's scores d_target [seqs,
        drafts + 1, vocab]: the accepted ones, one more token and -1 into d_token [seqs, drafts + 1] (int32), how many
        were accepted into d_accepted [seqs] (int32), and the tokens' log-probabilities under the target into
        d_logprob. d_draft [seqs, drafts, vocab]: the scores that the tokens were drawn from, of the target's type
        (None: they were not drawn); d_u [seqs, drafts + 1]: random numbers in [0, 1), a row's last one for the token
        after the accepted ones; draft_count [seqs] (int32): drafted tokens of each sequence; temperature [seqs]."""
        on = self._device
        if len(d_draft_token.shape) != 2:
            raise ValueError("d_draft_token is a 2-D tensor")
        seqs, drafts = d_draft_token.shape
        target, ld_target_seq, ld_target, vocab, dtype = _places(d_target, seqs, drafts + 1, "d_target", on)
        draft, ld_draft_seq, ld_draft = None, 0, 0
        if d_draft is not None:
            draft, ld_draft_seq, ld_draft, draft_vocab, draft_dtype = _places(d_draft, seqs, drafts, "d_draft", on)
            _same(draft_vocab, vocab, "the vocabulary of d_draft")
            if draft_dtype != dtype:
                raise TypeError(f"d_draft is {d_draft.dtype}, d_target {d_target.dtype}")
        places = seqs * (drafts + 1)
        self._check(self.lib.verify_dev(self._h, target, ld_target_seq, ld_target, draft, ld_draft_seq, ld_draft, dtype,
                                        seqs, _int(drafts, 32), vocab,
                                        _vector(d_draft_token, seqs * drafts, "d_draft_token", on, RBF_DTYPE_I32),
                                        _vector(draft_count, seqs, "draft_count", on, RBF_DTYPE_I32),
                                        _vector(d_u, places, "d_u", on, optional=False),
                                        _vector(temperature, seqs, "temperature", on),
                                        _vector(d_token, places, "d_token", on, RBF_DTYPE_I32, optional=False),
                                        _vector(d_accepted, seqs, "d_accepted", on, RBF_DTYPE_I32, optional=False),
                                        _vector(d_logprob, places, "d_logprob", on)), "verify_dev")

    def distill_dev(self, d_scores, d_index, d_teacher, d_loss=None, d_grad=None, rest=None, weight=None,
                    temperature: float = 1.0) -> None:
        """The loss of each row of d_scores [rows, vocab] against a teacher's best logits d_teacher [rows, k] at the
        indices d_index [rows, k] (int32; -1: no entry) into d_loss [rows], and the gradient of the losses' sum into
        d_grad [rows, vocab] (of d_scores' type). rest [rows]: the logarithm of the teacher's remaining mass at the
        temperature (None: none); weight [rows]: what each loss is multiplied by (None: 1), so a backward pass gives
        its loss' gradient and asks for d_grad alone."""
        on = self._device
        scores, ld_scores, rows, vocab, dtype = _float_matrix(d_scores, "d_scores", on)
        teacher, ld_teacher, t_rows, k, teacher_dtype = _float_matrix(d_teacher, "d_teacher", on)
        _same(t_rows, rows, "the number of rows of d_teacher")
        if _DTYPES.get(d_index.dtype) != RBF_DTYPE_I32:
            raise TypeError(f"d_index is {d_index.dtype}: expected int32")
        index, ld_index, i_rows, i_cols = _matrix(d_index, "d_index", on)
        _same((i_rows, i_cols), (rows, k), "the shape of d_index")
        grad, ld_grad = None, 0
        if d_grad is not None:
            grad, ld_grad, g_rows, g_cols, grad_dtype = _float_matrix(d_grad, "d_grad", on)
            _same((g_rows, g_cols), (rows, vocab), "the shape of d_grad")
            if grad_dtype != dtype:
                raise TypeError(f"d_grad is {d_grad.dtype}, d_scores {d_scores.dtype}")
        self._check(self.lib.distill_dev(self._h, scores, dtype, ld_scores, rows, vocab, index, ld_index, teacher,
                                         teacher_dtype, ld_teacher, k, _vector(rest, rows, "rest", on),
                                         _vector(weight, rows, "weight", on), float(temperature),
                                         _vector(d_loss, rows, "d_loss", on), grad, ld_grad), "distill_dev")
