"""8-bit products whose second operand's rows do not start on 16-byte boundaries: contiguous rows of odd lengths, views
that start anywhere, and enough rows for several parts."""
import numpy as np
import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(512, 65536, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == 0


def operands(m, n, k, offset=0, seed=0):
    g = np.random.default_rng(seed)
    a, b = (g.integers(-128, 128, (r, k), dtype=np.int8) for r in (m, n))
    # What lies around the rows is not zero.
    flat = torch.full((offset + n * k + 64,), 77, dtype=torch.int8, device="cuda")
    flat[offset:offset + n * k] = torch.from_numpy(b).cuda().flatten()
    return a, b, torch.from_numpy(a).cuda(), flat[offset:offset + n * k].view(n, k)


# One row more than a part of 32 MB holds, a part of few rows, an offset of each residue that matters.
@pytest.mark.parametrize("m,n,k,offset", [(1, 33281, 1001, 0), (3, 40003, 1001, 3), (5, 33281, 1001, 1), (40, 70001, 999, 2), (300, 66561, 1003, 15),
                                          (2, 3001, 40, 8), (130, 513, 65535, 0), (7, 1030, 32767, 5), (64, 5000, 1000, 0)])
def test_sums_are_exact(ops, m, n, k, offset):
    a, b, da, db = operands(m, n, k, offset)
    out = torch.full((m, n + 3), 5, dtype=torch.int32, device="cuda")
    ops.matmul_i8_dev(da, None, db, None, out[:, :n])
    assert np.array_equal(out[:, :n].cpu().numpy(), ref.product_sums(a, b))
    assert bool((out[:, n:] == 5).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m", [1, 4, 6, 200])
def test_equals_the_aligned_product(ops, m, dtype):
    """Scales, bias and rounding are applied to the same sums in the same order: the bits are the aligned call's."""
    n, k = 70001, 1001
    a, b, da, db = operands(m, n, k, 1, seed=m)
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    sa, sb, bias = (torch.rand(r, generator=g, device="cuda") * s for r, s in ((m, 0.01), (n, 0.01), (n, 1.0)))
    pitched = torch.empty(n, 1008, dtype=torch.int8, device="cuda")[:, :k]
    pitched.copy_(db)
    x = torch.randn(m, k, generator=g, device="cuda").to(dtype)
    for pad in (0, 7):
        want, got = (torch.full((m, n + pad), 3, dtype=dtype, device="cuda")[:, :n] for _ in range(2))
        ops.matmul_i8_dev(da, sa, pitched, sb, want, bias=bias)
        ops.matmul_i8_dev(da, sa, db, sb, got, bias=bias)
        assert torch.equal(want, got)
        ops.linear_i8_dev(x, pitched, sb, want, bias=bias)
        ops.linear_i8_dev(x, db, sb, got, bias=bias)
        assert torch.equal(want, got)
