"""The 8-bit floating-point product at depths past the handle's max_depth and past 65,536 (include/rbf_ops.h,
matmul_f8_dev): the gradient of a head's input has the vocabulary for its depth."""
import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import more_ops_reference as ref
from tests.test_gpu_more_ops_together import Head
from tests.test_gpu_ops_f8_instances import rows8

pytestmark = pytest.mark.gpu
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def operands(m, n, k, a8, block_rows, pad_a, pad_b):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + k)
    blocks = -(-k // 128)
    a, b = rows8(g, m, k, a8, pad_a, 0), rows8(g, n, k, E4M3, pad_b, 0)
    a_scale = torch.exp(torch.randn(m, blocks, generator=g, device="cuda")) * 1e-3
    b_scale = torch.exp(torch.randn(-(-n // block_rows), blocks, generator=g, device="cuda")) * 1e-3
    return a, a_scale, b, b_scale


# a's rows on 16-byte boundaries, b's too or put on them 256 at a time
@pytest.mark.parametrize("m,n,k,pad_a,pad_b", [(40, 300, 100003, 13, 13), (5, 515, 65537, 15, 0), (300, 520, 128000, 0, 0), (128, 700, 131072, 0, 3),
                                               (1, 1, 200000, 0, 0), (1000, 2560, 70400, 0, 0), (2, 130, 1 << 20, 16, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_depth_of_a_vocabulary(m, n, k, pad_a, pad_b, dtype, block_rows):
    a, a_scale, b, b_scale = operands(m, n, k, E5M2, block_rows, pad_a, pad_b)
    out = torch.empty(m, n, dtype=dtype, device="cuda")
    with rbf.Ops(1024, 256, stream=torch.cuda.current_stream()) as o:
        o.matmul_f8_dev(a, a_scale, b, b_scale, out)
        assert o.check_device_error() == rbf.RBF_OK
    want, size = ref.product(a, a_scale, b, b_scale, block_rows)
    assert bool(((out.double() - want).abs() <= ref.product_error(size, k, dtype, want)).all())


def test_rows_that_the_workspace_does_not_hold_are_refused():
    with rbf.Ops(64, 256, stream=torch.cuda.current_stream()) as o:
        for m, n, k, pad_a, pad_b, fits in ((40, 30, 100003, 0, 13, False), (2, 30, 16001, 0, 15, True), (3, 30, 16001, 0, 15, False),
                                            (4, 300, 140001, 15, 0, False), (4, 300, 131071, 1, 0, True), (65, 30, 256, 0, 0, False)):
            a, a_scale, b, b_scale = operands(m, n, k, E4M3, 128, pad_a, pad_b)
            out = torch.full((m, n), 5.0, device="cuda")
            if fits:
                o.matmul_f8_dev(a, a_scale, b, b_scale, out)
                want, size = ref.product(a, a_scale, b, b_scale, 128)
                assert bool(((out.double() - want).abs() <= ref.product_error(size, k, torch.float32, want)).all())
                continue
            with pytest.raises(rbf.RbfError) as e:
                o.matmul_f8_dev(a, a_scale, b, b_scale, out)
            assert e.value.status == rbf.RBF_ERR_INVALID_VALUE and o.last_launches == 0
            assert bool((out == 5.0).all())


def test_gradient_of_a_distillation_over_a_large_vocabulary():
    """Scores, their loss' gradient, that in 8 bits, and the gradient of the head's input, on one handle of the head's depth."""
    with rbf.Ops(16, 64, stream=torch.cuda.current_stream()) as o:
        h = Head(o, 3, 2, 70400, 64, seed=6)
        h.learn()
        assert o.check_device_error() == rbf.RBF_OK
        dx, size = ref.product(h.grad8, h.grad_scale, h.wt8, h.wt_scale, 128)
        assert float(dx.abs().max()) > 0
        assert bool(((h.dx.double() - dx).abs() <= ref.product_error(size, h.vocab, torch.float32, dx)).all())
