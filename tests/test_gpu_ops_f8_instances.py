"""Every instance of the 8-bit floating-point product (include/rbf_ops.h, matmul_f8_dev): tiles of 32, 64, 128 and 256 tokens,
several whole tiles a pair of CTAs, and tiles whose stages several pairs share, each to all output types and with both kinds
of scales. What lies between the rows and behind them is NaN."""
import math

import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import more_ops_reference as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(1024, 16384, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == rbf.RBF_OK


def among_nan(t, pad, shift=0):
    """The matrix in rows of `pad` more elements, `shift` elements into an allocation that is NaN elsewhere."""
    rows, cols = t.shape
    flat = torch.full((rows * (cols + pad) + shift + 64,), 0x7F if t.dtype.itemsize == 1 else math.nan,
                      dtype=torch.uint8 if t.dtype.itemsize == 1 else t.dtype, device="cuda")
    flat = flat.view(t.dtype) if t.dtype.itemsize == 1 else flat
    out = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    out.copy_(t)
    return out


def rows8(g, rows, cols, dtype, pad, shift):
    top = ref.F8[dtype][0]
    return among_nan((torch.randn(rows, cols, generator=g, device="cuda") * (top / 3)).clamp_(-top, top).to(dtype), pad, shift)


def check(ops, m, n, k, dtype, block_rows, a8=E4M3, pad=0, shift=0, out_pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(m * 7 + n * 3 + k)
    blocks = -(-k // 128)
    a, b = rows8(g, m, k, a8, pad, shift), rows8(g, n, k, E4M3, pad, shift)
    small = 2.0 ** -7 if a8 == E5M2 else 1.0  # within fp16's range
    a_scale = among_nan(torch.exp(torch.randn(m, blocks, generator=g, device="cuda")) * small, pad % 5)
    b_scale = among_nan(torch.exp(torch.randn(-(-n // block_rows), blocks, generator=g, device="cuda")) * 1e-3, pad % 3)
    bias = torch.randn(n, generator=g, device="cuda")
    whole = torch.full((m + 1, n + out_pad), 5.0, dtype=dtype, device="cuda")
    out = whole[:m, :n]
    ops.matmul_f8_dev(a, a_scale, b, b_scale, out, bias=bias)
    want, size = ref.product(a, a_scale, b, b_scale, block_rows, bias)
    off, allowed = (out.double() - want).abs(), ref.product_error(size, k, dtype, want)
    fine = off <= allowed
    if dtype == torch.float16:  # 65,520 and above round to infinity
        fine |= (out.double() == want.sign() * math.inf) & (want.abs() + allowed >= 65520.0)
    assert bool(fine.all()), float((off / allowed).max())
    assert bool((whole[m:] == 5.0).all()) and bool((whole[:, n:] == 5.0).all())
    again = torch.empty_like(out)
    for _ in range(3):
        ops.matmul_f8_dev(a, a_scale, b, b_scale, again, bias=bias)
        assert torch.equal(again, out)


TYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
SCALES = pytest.mark.parametrize("block_rows", [1, 128])


@pytest.mark.parametrize("m,n,k,pad,out_pad", [(8, 40011, 200, 56, 5), (64, 40011, 200, 8, 0), (128, 40016, 130, 14, 0), (513, 20011, 300, 4, 5),
                                               (1000, 2560, 300, 20, 0), (1000, 20011, 300, 4, 5), (900, 20011, 128, 0, 2)])
@TYPES
@SCALES
def test_whole_tiles(ops, m, n, k, pad, out_pad, dtype, block_rows):
    """More tiles than pairs (76 on 152 SMs), of 32, 64 and 128 tokens; 256 from the fourth size on but for the 513 tokens."""
    check(ops, m, n, k, dtype, block_rows, pad=pad, out_pad=out_pad)


@pytest.mark.parametrize("m,n,k,pad,out_pad", [(8, 1000, 8192, 16, 0), (40, 1003, 8192, 0, 5), (100, 1000, 8100, 12, 0), (128, 1027, 8192, 32, 1),
                                               (1000, 2560, 16384, 16, 8)])
@TYPES
@SCALES
def test_shared_tiles(ops, m, n, k, pad, out_pad, dtype, block_rows):
    """Fewer tiles than pairs and many stages: tiles of 32, 64, 128, 128 and 256 tokens are summed from pairs' partial sums."""
    check(ops, m, n, k, dtype, block_rows, pad=pad, out_pad=out_pad)


@pytest.mark.parametrize("m,n,k", [(40, 3001, 700), (1000, 2560, 390)])
@TYPES
@SCALES
def test_types_and_rows_off_boundaries(ops, m, n, k, dtype, block_rows):
    check(ops, m, n, k, dtype, block_rows, a8=E5M2, pad=3, shift=5, out_pad=3)
