"""Refusals of the 8-bit floating-point, verification and distillation operators, on the CPU: the binding refuses
misshapen, mistyped and overlapping arguments before any pointer reaches the library, and the C entry points refuse
without a handle."""
import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests.test_ops_checks import _Cuda, _On, f32, i32, i8, ops  # noqa: F401

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def f8(*shape, dtype=E4M3):
    return _Cuda(torch.zeros(*shape).to(dtype))


def f16(*shape):
    return _Cuda(torch.zeros(*shape, dtype=torch.float16))


def verify(o, target=None, tokens=None, u=None, token=None, accepted=None, **more):
    o.verify_dev(f32(2, 4, 9) if target is None else target, i32(2, 3) if tokens is None else tokens, f32(2, 4) if u is None else u,
                 i32(2, 4) if token is None else token, i32(2) if accepted is None else accepted, **more)


def distill(o, scores=None, index=None, teacher=None, **more):
    o.distill_dev(f32(3, 9) if scores is None else scores, i32(3, 2) if index is None else index, f32(3, 2) if teacher is None else teacher, **more)


@pytest.mark.parametrize("call", [
    lambda o: o.quantize_f8_dev(f32(3, 4), f8(3, 5), f32(3, 1)),
    lambda o: o.quantize_f8_dev(f32(3, 4), f8(3, 4), f32(3)),
    lambda o: o.quantize_f8_dev(f32(3, 4), f8(3, 4), f32(3, 2)),
    lambda o: o.quantize_f8_dev(f32(3, 4), f8(3, 4), f32(3, 1), block_rows=128),
    lambda o: o.quantize_f8_dev(f32(3, 4), f8(3, 4), f32(3, 1), block_rows=2),
    lambda o: o.quantize_f8_dev(_Cuda(torch.zeros(4, 3).t()), f8(3, 4), f32(3, 1)),
    lambda o: o.quantize_f8_dev(_Cuda(torch.zeros(1, 4).expand(3, 4)), f8(3, 4), f32(3, 1)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(3, 9), f32(3, 1), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(3, 8), f32(3, 1), f32(3, 2)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(3, 1), f8(3, 8), f32(3, 1), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 2), f8(3, 8), f32(3, 1), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(3, 8), f32(2, 1), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(130, 8), f32(3, 1), f32(2, 130)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(3, 8), f32(3), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(3, 8), f32(3, 1), f32(2, 3), bias=f32(4)),
    lambda o: verify(o, target=f32(2, 3, 9)),
    lambda o: verify(o, target=f32(3, 4, 9)),
    lambda o: verify(o, target=f32(8, 9)),
    lambda o: verify(o, target=_Cuda(torch.zeros(2, 9, 4).transpose(1, 2))),
    lambda o: verify(o, target=_Cuda(torch.zeros(2, 1, 9).expand(2, 4, 9))),
    lambda o: verify(o, target=_Cuda(torch.zeros(1, 4, 9).expand(2, 4, 9))),
    lambda o: verify(o, tokens=i32(6)),
    lambda o: verify(o, u=f32(2, 3)),
    lambda o: verify(o, token=i32(2, 3)),
    lambda o: verify(o, accepted=i32(3)),
    lambda o: verify(o, d_draft=f32(2, 4, 9)),
    lambda o: verify(o, d_draft=f32(2, 3, 8)),
    lambda o: verify(o, d_draft=_Cuda(torch.zeros(1, 3, 9).expand(2, 3, 9))),
    lambda o: verify(o, draft_count=i32(3)),
    lambda o: verify(o, temperature=f32(1)),
    lambda o: verify(o, d_logprob=f32(2)),
    lambda o: distill(o, index=i32(3, 1)),
    lambda o: distill(o, index=i32(2, 2)),
    lambda o: distill(o, teacher=f32(2, 2)),
    lambda o: distill(o, scores=f32(9)),
    lambda o: distill(o, d_loss=f32(2)),
    lambda o: distill(o, d_grad=f32(3, 8)),
    lambda o: distill(o, rest=f32(2)),
    lambda o: distill(o, weight=f32(9)),
    lambda o: distill(o, d_grad=_Cuda(torch.zeros(1, 9).expand(3, 9))),
])
def test_shapes_are_refused(ops, call):  # noqa: F811
    with pytest.raises(ValueError):
        call(ops)


@pytest.mark.parametrize("call", [
    lambda o: o.quantize_f8_dev(i8(3, 4), f8(3, 4), f32(3, 1)),
    lambda o: o.quantize_f8_dev(f32(3, 4), i8(3, 4), f32(3, 1)),
    lambda o: o.quantize_f8_dev(f32(3, 4), f8(3, 4), f16(3, 1)),
    lambda o: o.quantize_f8_dev(torch.zeros(3, 4), f8(3, 4), f32(3, 1)),
    lambda o: o.matmul_f8_dev(i8(2, 8), f32(2, 1), f8(3, 8), f32(3, 1), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f32(3, 8), f32(3, 1), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f16(2, 1), f8(3, 8), f32(3, 1), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(3, 8), i32(3, 1), f32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(3, 8), f32(3, 1), i32(2, 3)),
    lambda o: o.matmul_f8_dev(f8(2, 8), f32(2, 1), f8(3, 8), f32(3, 1), f32(2, 3), bias=f16(3)),
    lambda o: verify(o, target=i32(2, 4, 9)),
    lambda o: verify(o, target=torch.zeros(2, 4, 9)),
    lambda o: verify(o, tokens=f32(2, 3)),
    lambda o: verify(o, token=f32(2, 4)),
    lambda o: verify(o, d_draft=f16(2, 3, 9)),
    lambda o: verify(o, draft_count=f32(2)),
    lambda o: distill(o, scores=i32(3, 9)),
    lambda o: distill(o, index=f32(3, 2)),
    lambda o: distill(o, teacher=i32(3, 2)),
    lambda o: distill(o, d_grad=f16(3, 9)),
    lambda o: distill(o, weight=f16(3)),
])
def test_types_are_refused(ops, call):  # noqa: F811
    with pytest.raises(TypeError):
        call(ops)


def test_c_entry_points_refuse_without_a_handle():
    from resident_brute_force_gb300 import _build
    _build.build()
    lib = rbf.load_library()
    bad = rbf.RBF_ERR_INVALID_VALUE
    assert lib.quantize_f8_dev(None, 16, 0, 4, 1, 4, 1, 16, 5, 4, 16, 1) == bad
    assert lib.matmul_f8_dev(None, 16, 5, 4, 16, 1, 16, 5, 4, 16, 1, 1, None, 16, 0, 4, 1, 4, 4) == bad
    assert lib.verify_dev(None, 16, 4, 4, None, 0, 0, 0, 1, 0, 4, None, None, 16, None, 16, 16, None) == bad
    assert lib.distill_dev(None, 16, 0, 4, 1, 4, 16, 1, 16, 0, 1, 1, None, None, 1.0, 16, None, 0) == bad


F = torch.float32
CALLS = {
    "quantize_f8_dev": [("d_x", (3, 4), F), ("d_q", (3, 4), E4M3), ("d_scale", (3, 1), F)],
    "matmul_f8_dev": [("d_a", (2, 8), E4M3), ("d_a_scale", (2, 1), F), ("d_b", (3, 8), E5M2), ("d_b_scale", (3, 1), F), ("d_out", (2, 3), F),
                      ("bias", (3,), F)],
    "verify_dev": [("d_target", (2, 4, 9), F), ("d_draft_token", (2, 3), torch.int32), ("d_u", (2, 4), F), ("d_token", (2, 4), torch.int32),
                   ("d_accepted", (2,), torch.int32), ("d_logprob", (2, 4), F), ("d_draft", (2, 3, 9), F), ("draft_count", (2,), torch.int32),
                   ("temperature", (2,), F)],
    "distill_dev": [("d_scores", (3, 9), F), ("d_index", (3, 2), torch.int32), ("d_teacher", (3, 2), F), ("d_loss", (3,), F), ("d_grad", (3, 9), F),
                    ("rest", (3,), F), ("weight", (3,), F)],
}


@pytest.mark.parametrize("call,other", [(call, a[0]) for call, args in CALLS.items() for a in args])
def test_tensors_of_another_device_are_refused(ops, call, other):  # noqa: F811
    ops._device = 1
    args = {name: _On(torch.zeros(shape).to(dtype), 0 if name == other else 1) for name, shape, dtype in CALLS[call]}
    with pytest.raises(ValueError, match="device"):
        getattr(ops, call)(**args)


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_the_handles_device_pass(ops, call):  # noqa: F811
    ops._device = 1
    with pytest.raises(AssertionError, match="reached the library"):
        getattr(ops, call)(**{name: _On(torch.zeros(shape).to(dtype), 1) for name, shape, dtype in CALLS[call]})


@pytest.mark.parametrize("cols", [2 ** 31, 2 ** 32 + 8])
@pytest.mark.parametrize("call,wide", [("quantize_f8_dev", ("d_x", "d_q")), ("matmul_f8_dev", ("d_a", "d_b")), ("verify_dev", ("d_target", "d_draft")),
                                       ("distill_dev", ("d_scores", "d_grad")), ("distill_dev", ("d_index", "d_teacher"))])
def test_rows_past_31_bits_are_refused(ops, call, wide, cols):  # noqa: F811
    args = {}
    for name, shape, dtype in CALLS[call]:
        args[name] = _Cuda(torch.empty((*shape[:-1], cols) if name in wide else shape, dtype=dtype, device="meta"))
    with pytest.raises(ValueError, match="2\\^31"):
        getattr(ops, call)(**args)
