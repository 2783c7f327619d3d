"""Refusals of the scoring-head operators, on the CPU: the binding refuses
misshapen, mistyped and overlapping arguments before any pointer reaches the
library, and the C entry points refuse bad sizes without a GPU call."""
import ctypes

import pytest
import torch

import resident_brute_force_gb300 as rbf
from resident_brute_force_gb300 import ops as binding


class _Cuda:
    """A tensor's shape, type and strides with is_cuda set, for checks that come before any use of the data."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True
        self.shape, self.dtype = t.shape, t.dtype

    def __getattr__(self, name):
        return getattr(self._t, name)


class _NoLibrary:
    def __getattr__(self, name):
        def reached(*args):
            raise AssertionError(f"{name} reached the library")
        return reached


@pytest.fixture
def ops():
    o = object.__new__(rbf.Ops)
    o.lib, o._h = _NoLibrary(), None
    return o


def i8(*shape):
    return _Cuda(torch.zeros(*shape, dtype=torch.int8))


def f32(*shape):
    return _Cuda(torch.zeros(*shape))


def i32(*shape):
    return _Cuda(torch.zeros(*shape, dtype=torch.int32))


@pytest.mark.parametrize("call", [
    lambda o: o.quantize_rows_i8_dev(f32(3, 4), i8(3, 5), f32(3)),
    lambda o: o.quantize_rows_i8_dev(f32(3, 4), i8(3, 4), f32(2)),
    lambda o: o.quantize_rows_i8_dev(f32(12), i8(3, 4), f32(3)),
    lambda o: o.quantize_rows_i8_dev(f32(3, 4), i8(3, 4), None),
    lambda o: o.quantize_rows_i8_dev(_Cuda(torch.zeros(4, 3).t()), i8(3, 4), f32(3)),
    lambda o: o.quantize_rows_i8_dev(_Cuda(torch.zeros(1, 4).expand(3, 4)), i8(3, 4), f32(3)),
    lambda o: o.matmul_i8_dev(i8(2, 8), None, i8(3, 9), None, f32(2, 3)),
    lambda o: o.matmul_i8_dev(i8(2, 8), None, i8(3, 8), None, f32(3, 2)),
    lambda o: o.matmul_i8_dev(i8(2, 8), f32(3), i8(3, 8), None, f32(2, 3)),
    lambda o: o.matmul_i8_dev(i8(2, 8), None, i8(3, 8), f32(2), f32(2, 3)),
    lambda o: o.matmul_i8_dev(i8(2, 8), None, i8(3, 8), None, f32(2, 3), bias=f32(4)),
    lambda o: o.linear_i8_dev(f32(2, 8), i8(3, 7), None, f32(2, 3)),
    lambda o: o.linear_i8_dev(f32(2, 8), i8(3, 8), None, f32(2, 4)),
    lambda o: o.sample_dev(f32(2, 8), f32(3), i32(2)),
    lambda o: o.sample_dev(f32(2, 8), f32(2), i32(3)),
    lambda o: o.sample_dev(f32(2, 8), None, i32(2)),
    lambda o: o.sample_dev(f32(2, 8), f32(2), i32(2), f32(1)),
    lambda o: o.sample_dev(f32(2, 8), f32(2), i32(2), top_k=i32(1)),
    lambda o: o.sample_dev(f32(16), f32(2), i32(2)),
])
def test_shapes_are_refused(ops, call):
    with pytest.raises(ValueError):
        call(ops)


@pytest.mark.parametrize("call", [
    lambda o: o.quantize_rows_i8_dev(i8(3, 4), i8(3, 4), f32(3)),
    lambda o: o.quantize_rows_i8_dev(f32(3, 4), f32(3, 4), f32(3)),
    lambda o: o.quantize_rows_i8_dev(torch.zeros(3, 4), i8(3, 4), f32(3)),
    lambda o: o.matmul_i8_dev(f32(2, 8), None, i8(3, 8), None, f32(2, 3)),
    lambda o: o.matmul_i8_dev(i8(2, 8), None, f32(3, 8), None, f32(2, 3)),
    lambda o: o.matmul_i8_dev(i8(2, 8), None, i8(3, 8), None, i8(2, 3)),
    lambda o: o.linear_i8_dev(i8(2, 8), i8(3, 8), None, f32(2, 3)),
    lambda o: o.linear_i8_dev(f32(2, 8), i8(3, 8), None, i32(2, 3)),
    lambda o: o.sample_dev(i32(2, 8), f32(2), i32(2)),
    lambda o: o.sample_dev(f32(2, 8), f32(2), f32(2)),
    lambda o: o.sample_dev(f32(2, 8), f32(2), i32(2), top_k=f32(2)),
])
def test_types_are_refused(ops, call):
    with pytest.raises(TypeError):
        call(ops)


def test_c_entry_points_refuse_without_a_handle():
    from resident_brute_force_gb300 import _build
    _build.build()
    lib = rbf.load_library()
    bad = rbf.RBF_ERR_INVALID_VALUE
    assert lib.rbf_ops_create(1, 1, None, None) == bad
    h = ctypes.c_void_p()
    for rows, depth in ((0, 1), (1, 0), (-1, 5), ((1 << 20) + 1, 1), (1, binding.RBF_OPS_MAX_DEPTH + 1)):
        assert lib.rbf_ops_create(rows, depth, None, ctypes.byref(h)) == bad and not h.value
    assert lib.rbf_ops_destroy(None) == rbf.RBF_OK
    assert lib.rbf_ops_check_device_error(None) == bad
    assert lib.quantize_rows_i8_dev(None, 16, 0, 4, 1, 4, 16, 4, 16) == bad
    assert lib.matmul_i8_dev(None, 16, 4, None, 16, 4, None, None, 16, 0, 4, 1, 4, 4) == bad
    assert lib.linear_i8_dev(None, 16, 0, 4, 16, 4, None, None, 16, 0, 4, 1, 4, 4) == bad
    assert lib.sample_dev(None, 16, 0, 4, 1, 4, 16, None, None, None, None, 16, None) == bad


class _On(_Cuda):
    """A stand-in on a device of its own."""

    def __init__(self, t, device):
        super().__init__(t)
        self._device = device

    def get_device(self):
        return self._device


CALLS = {
    "quantize_rows_i8_dev": [("d_x", (3, 4), torch.float32), ("d_q", (3, 4), torch.int8), ("d_scale", (3,), torch.float32)],
    "matmul_i8_dev": [("d_a", (2, 8), torch.int8), ("d_a_scale", (2,), torch.float32), ("d_b", (3, 8), torch.int8),
                      ("d_b_scale", (3,), torch.float32), ("d_out", (2, 3), torch.float32), ("bias", (3,), torch.float32)],
    "linear_i8_dev": [("d_x", (2, 8), torch.float32), ("d_w", (3, 8), torch.int8), ("d_w_scale", (3,), torch.float32),
                      ("d_out", (2, 3), torch.float32), ("bias", (3,), torch.float32)],
    "sample_dev": [("d_logits", (2, 8), torch.float32), ("d_u", (2,), torch.float32), ("d_token", (2,), torch.int32),
                   ("d_logprob", (2,), torch.float32), ("temperature", (2,), torch.float32), ("top_k", (2,), torch.int32),
                   ("top_p", (2,), torch.float32), ("min_p", (2,), torch.float32)],
}


@pytest.mark.parametrize("call,other", [(call, a[0]) for call, args in CALLS.items() for a in args])
def test_tensors_of_another_device_are_refused(ops, call, other):
    ops._device = 1
    args = {name: _On(torch.zeros(shape, dtype=dtype), 0 if name == other else 1) for name, shape, dtype in CALLS[call]}
    with pytest.raises(ValueError, match="device"):
        getattr(ops, call)(**args)


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_the_handles_device_pass(ops, call):
    ops._device = 1
    with pytest.raises(AssertionError, match="reached the library"):
        getattr(ops, call)(**{name: _On(torch.zeros(shape, dtype=dtype), 1) for name, shape, dtype in CALLS[call]})


@pytest.mark.parametrize("cols", [2 ** 31, 2 ** 32, 2 ** 32 + 8])
@pytest.mark.parametrize("call", CALLS)
def test_rows_past_31_bits_are_refused(ops, call, cols):
    """Not cut to their low 32 bits on the way to the library."""
    args = {}
    for name, shape, dtype in CALLS[call]:
        if name in ("d_x", "d_q", "d_a", "d_b", "d_w", "d_logits"):
            shape = (shape[0], cols)
        args[name] = _Cuda(torch.empty(shape, dtype=dtype, device="meta"))
    with pytest.raises(ValueError, match="2\\^31"):
        getattr(ops, call)(**args)


@pytest.mark.parametrize("size,as_passed", [((1, 2 ** 32 + 64), (1, 2 ** 31 - 1)), ((2 ** 64 + 4, 64), (2 ** 63 - 1, 64)),
                                            ((1, -(2 ** 32) + 64), (1, -(2 ** 31))), ((4, 64), (4, 64))])
def test_handle_sizes_reach_the_library_as_they_are(monkeypatch, size, as_passed):
    """A size past what the library's type holds is passed as one that it refuses."""
    import types
    seen = []

    def create(rows, depth, stream, out):
        seen.append((rows, depth))
        return rbf.RBF_ERR_INVALID_VALUE

    monkeypatch.setattr(binding, "load_library", lambda: types.SimpleNamespace(rbf_ops_create=create))
    with pytest.raises(rbf.RbfError):
        rbf.Ops(*size)
    assert seen == [as_passed]
