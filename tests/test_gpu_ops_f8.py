"""8-bit floating-point rows and their product (include/rbf_ops.h) against the definition in 64 bits."""
import math

import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import more_ops_reference as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(4096, 8192, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == rbf.RBF_OK


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def pitched(rows, cols, dtype, pad=0, shift=0):
    """[rows, cols] in rows of cols + pad, `shift` elements into the allocation."""
    flat = torch.zeros(rows * (cols + pad) + shift, dtype=torch.uint8 if dtype.itemsize == 1 else dtype, device="cuda")[shift:]
    flat = flat.view(dtype) if dtype.itemsize == 1 else flat
    return flat.view(rows, cols + pad)[:, :cols]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("f8", [E4M3, E5M2])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (1, 768, 0, 0), (3, 127, 1, 0), (130, 129, 0, 0), (128, 256, 8, 1),
                                                 (257, 1000, 3, 5), (300, 384, 16, 0)])
def test_quantize(ops, dtype, f8, block_rows, rows, cols, pad, shift):
    g = gen(rows * cols + pad)
    x = pitched(rows, cols, dtype, pad, shift)
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(torch.randn(rows, 1, generator=g, device="cuda")))
    q = pitched(rows, cols, f8, pad, shift)
    scale = torch.empty(-(-rows // block_rows), -(-cols // 128), device="cuda")
    ops.quantize_f8_dev(x, q, scale, block_rows=block_rows)
    want, want_scale = ref.quantize_f8(x, f8, block_rows)
    assert torch.equal(q.double(), want)
    assert torch.equal(scale, want_scale)


def test_quantize_special_blocks(ops):
    x = torch.randn(8, 512, generator=gen(3), device="cuda")
    x[0, :128] = 0
    x[1, 130] = math.nan
    x[2, 300] = math.inf
    x[3, 5] = -math.inf
    x[4, :128] *= 1e-38  # MAX / t overflows
    x[5, 128:256] = 1e-45
    x[6, :] *= 1e37
    x[7, 256:384] = 0
    x[7, 256] = -2.0 ** 127
    for f8 in (E4M3, E5M2):
        for block_rows in (1, 128):
            q, scale = torch.empty(8, 512, dtype=f8, device="cuda"), torch.empty(8 if block_rows == 1 else 1, 4, device="cuda")
            ops.quantize_f8_dev(x, q, scale, block_rows=block_rows)
            want, want_scale = ref.quantize_f8(x, f8, block_rows)
            assert torch.equal(q.double(), want)
            assert torch.equal(scale.isnan(), want_scale.isnan()) and torch.equal(scale.nan_to_num(), want_scale.nan_to_num())
            assert not torch.isnan(q.double()).any()


def test_quantize_leaves_the_rest(ops):
    whole = torch.full((10, 200), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((12, 5), -1.0, device="cuda")
    x = torch.randn(8, 150, generator=gen(4), device="cuda")
    ops.quantize_f8_dev(x, whole[1:9, 8:158].view(E4M3), scales[2:10, 1:3])
    keep = torch.ones_like(whole, dtype=torch.bool)
    keep[1:9, 8:158] = False
    assert bool((whole[keep] == 7).all())
    keep = torch.ones_like(scales, dtype=torch.bool)
    keep[2:10, 1:3] = False
    assert bool((scales[keep] == -1.0).all())


def operands(g, m, n, k, a8, b8, block_rows, pad=0, shift=0):
    a, b = pitched(m, k, a8, pad, shift), pitched(n, k, b8, pad, shift)
    for t, kind in ((a, a8), (b, b8)):
        top = ref.F8[kind][0]
        t.copy_((torch.randn(t.shape, generator=g, device="cuda") * (top / 3)).clamp_(-top, top))
    blocks = -(-k // 128)
    a_scale = torch.exp(torch.randn(m, blocks, generator=g, device="cuda"))
    b_scale = torch.exp(torch.randn(-(-n // block_rows), blocks, generator=g, device="cuda")) * 1e-3
    return a, a_scale, b, b_scale


def check_product(ops, m, n, k, a8=E4M3, b8=E4M3, block_rows=1, dtype=torch.float32, with_bias=False, pad=0, shift=0, out_pad=0, factor=1.0):
    g = gen(m * 7 + n * 3 + k)
    a, a_scale, b, b_scale = operands(g, m, n, k, a8, b8, block_rows, pad, shift)
    b_scale *= factor
    bias = torch.randn(n, generator=g, device="cuda") if with_bias else None
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
    ops.matmul_f8_dev(a, a_scale, b, b_scale, again, bias=bias)
    assert torch.equal(again, out)


SIZES = [(1, 1, 1), (1, 130, 64), (1, 1000, 4096), (2, 257, 128), (3, 100, 129), (5, 384, 1000), (8, 4000, 512), (16, 513, 2048), (33, 255, 384),
         (64, 1024, 256), (100, 1000, 1000), (128, 128, 128), (129, 300, 640), (200, 257, 768), (256, 2048, 256), (257, 1111, 130), (700, 900, 1024)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_product_sizes(ops, m, n, k, block_rows):
    check_product(ops, m, n, k, block_rows=block_rows)


@pytest.mark.parametrize("m,n,k", [(1, 700, 384), (4, 300, 256), (40, 517, 1000), (300, 520, 512)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("a8,b8", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
def test_product_types(ops, m, n, k, dtype, a8, b8):
    small = sum(t == E5M2 for t in (a8, b8)) if dtype == torch.float16 else 0  # such sums pass fp16's range
    check_product(ops, m, n, k, a8, b8, 1 if dtype == torch.float32 else 128, dtype, with_bias=True, factor=2.0 ** (-7 * small))


@pytest.mark.parametrize("m,n,k,pad,shift,out_pad", [(1, 300, 385, 0, 0, 0), (3, 257, 200, 3, 1, 1), (60, 300, 385, 0, 0, 3), (150, 300, 1001, 7, 5, 0),
                                                     (300, 264, 256, 16, 16, 8), (31, 1000, 129, 0, 3, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product_strides(ops, m, n, k, pad, shift, out_pad, dtype):
    check_product(ops, m, n, k, block_rows=128, dtype=dtype, pad=pad, shift=shift, out_pad=out_pad)


def test_product_scale_strides(ops):
    g = gen(11)
    a, a_scale, b, b_scale = operands(g, 70, 300, 640, E4M3, E4M3, 128)
    wide_a, wide_b = torch.full((70, 9), math.nan, device="cuda"), torch.full((3, 11), math.nan, device="cuda")
    wide_a[:, 2:7], wide_b[:, 3:8] = a_scale, b_scale
    out, want = torch.empty(70, 300, device="cuda"), torch.empty(70, 300, device="cuda")
    ops.matmul_f8_dev(a, a_scale, b, b_scale, want)
    ops.matmul_f8_dev(a, wide_a[:, 2:7], b, wide_b[:, 3:8], out)
    assert torch.equal(out, want)


def test_product_exact_on_whole_numbers(ops):
    """Small whole numbers and scales that are powers of two: every sum is exact, whatever the order."""
    for m, n, k in ((1, 513, 1000), (7, 300, 256), (130, 270, 4096)):
        g = gen(m)
        a = torch.randint(-8, 9, (m, k), generator=g, device="cuda").to(E4M3)
        b = torch.randint(-8, 9, (n, k), generator=g, device="cuda").to(E4M3)
        blocks = -(-k // 128)
        a_scale = torch.exp2(torch.randint(-1, 2, (m, blocks), generator=g, device="cuda").float())
        b_scale = torch.exp2(torch.randint(-1, 2, (n, blocks), generator=g, device="cuda").float())
        out = torch.empty(m, n, device="cuda")
        ops.matmul_f8_dev(a, a_scale, b, b_scale, out)
        assert torch.equal(out.double(), ref.product(a, a_scale, b, b_scale, 1)[0])


@pytest.mark.parametrize("m", [1, 3, 20, 140])
def test_product_nan_and_infinity_stay_in_their_rows(ops, m):
    n, k = 300, 384
    g = gen(m)
    a, a_scale, b, b_scale = operands(g, m, n, k, E5M2, E5M2, 1)
    a_scale, b_scale = a_scale * 1e-4, b_scale * 1e-4
    want, size = ref.product(a, a_scale, b, b_scale, 1)
    a[m - 1, 130] = math.inf
    b[7, 5] = math.nan
    b_scale[9, 2] = math.nan
    out = torch.empty(m, n, device="cuda")
    ops.matmul_f8_dev(a, a_scale, b, b_scale, out)
    assert bool(out[:, 7].isnan().all()) and bool(out[:, 9].isnan().all()) and not bool(torch.isfinite(out[m - 1]).any())
    cols = [j for j in range(n) if j not in (7, 9)]
    off = (out[:m - 1].double() - want[:m - 1]).abs()[:, cols]
    assert bool((off <= ref.product_error(size, k, torch.float32, want)[:m - 1][:, cols]).all())


def test_product_of_no_depth_and_empty(ops):
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    out, bias = torch.full((3, 5), 9.0, device="cuda"), torch.arange(5.0, device="cuda")
    ops.matmul_f8_dev(e(3, 0).to(E4M3), e(3, 0), e(5, 0).to(E4M3), e(5, 0), out, bias=bias)
    assert torch.equal(out, bias.expand(3, 5))
    ops.matmul_f8_dev(e(0, 64).to(E4M3), e(0, 1), e(5, 64).to(E4M3), e(5, 1), e(0, 5))
    assert ops.last_launches == 0
    ops.quantize_f8_dev(e(0, 64), e(0, 64).to(E4M3), e(0, 1))
    assert ops.last_launches == 0


def test_linear_layer_gradients(ops):
    """Forward and both gradients of y = x w^T by three products, each operand quantised along the depth it is summed
    over, against 64 bits: a quantised value is off by half a step of its mantissa, or of its block's smallest number."""
    g = gen(5)
    m, n, k = 160, 200, 300
    x, w, dy = (torch.randn(*s, generator=g, device="cuda") for s in ((m, k), (n, k), (m, n)))

    def quantised(t, f8):
        q, scale = torch.empty(t.shape, dtype=f8, device="cuda"), torch.empty(t.shape[0], -(-t.shape[1] // 128), device="cuda")
        ops.quantize_f8_dev(t.contiguous(), q, scale)
        step = 2.0 ** -4 if f8 == E4M3 else 2.0 ** -3
        low = scale.double().repeat_interleave(128, 1)[:, :t.shape[1]] * (2.0 ** -10 if f8 == E4M3 else 2.0 ** -17)
        return q, scale, t.double().abs() * step + low

    for p, q, p8 in ((x, w, E4M3), (dy, w.t(), E5M2), (dy.t(), x.t(), E5M2)):
        p8, ps, pe = quantised(p, p8)
        q8, qs, qe = quantised(q, E4M3)
        out = torch.empty(p.shape[0], q.shape[0], device="cuda")
        ops.matmul_f8_dev(p8, ps, q8, qs, out)
        allowed = pe @ q.double().abs().t() + p.double().abs() @ qe.t() + pe @ qe.t()
        assert bool(((out.double() - p.double() @ q.double().t()).abs() <= allowed * 1.001).all())
