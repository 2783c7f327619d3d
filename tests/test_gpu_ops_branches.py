"""The scoring-head operators on the inputs that take a kernel of their own or a branch of it: depths past 8,192, tokens
that fill most of shared memory, tiles shared by CTA pairs whose outputs end inside 16 bytes, special values in 16-bit
rows, and rows of scores too long for a cluster's shared memory."""
import numpy as np
import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import ops_reference as ref
from tests.test_gpu_ops import FLOATS, ROUNDING, check_allowed, check_exact, on_gpu, run_quantize, run_sample, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(1024, 65536, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == rbf.RBF_OK


def integers(seed, rows, cols, pitch=16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.empty(rows, -(-cols // pitch) * pitch, dtype=torch.int8, device="cuda")
    t.copy_(torch.randint(-128, 128, t.shape, generator=g, device="cuda", dtype=torch.int8))
    return t[:, :cols]


def sums(a, b):
    """Exact: 64-bit floats hold every sum (under 2^53)."""
    return torch.mm(a.double(), b.double().t())


def check(out, exact, a_scale, b_scale, bias):
    """One rounding to the output's type, three in fp32 and one of the bias, as in the tests of the product."""
    scaled = exact * a_scale.double()[:, None] * b_scale.double()
    want = scaled + bias.double()
    room = ROUNDING[out.dtype] * want.abs() + 4 * 2.0 ** -24 * (scaled.abs() + want.abs()) + (2.0 ** -25 if out.dtype == torch.float16 else 0)
    off = (out.double() - want).abs()
    assert bool((off <= room).all()), off.max()


# (tokens, rows, depth): more than 48 KB of tokens, the most that fit, and one row more; one deep row.
@pytest.mark.parametrize("m,n,k", [(4, 3001, 16384), (3, 5003, 32768), (4, 700, 32768), (1, 3001, 65536), (2, 20011, 40000), (1, 257, 65535)])
def test_few_deep_tokens(ops, m, n, k):
    a, b = integers(m, m, k), integers(n, n, k)
    out = torch.empty(m, n, dtype=torch.int32, device="cuda")
    ops.matmul_i8_dev(a, None, b, None, out)
    assert torch.equal(out.double(), sums(a, b))
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    scale, bias = torch.rand(n, generator=g, device="cuda") * 0.01, torch.randn(n, generator=g, device="cuda")
    for dtype in FLOATS.values():
        x = torch.randn(m, k, generator=g, device="cuda").to(dtype)
        q, s = ref.quantize(x.float().cpu().numpy())
        out = torch.empty(m, n, dtype=dtype, device="cuda")
        ops.linear_i8_dev(x, b, scale, out, bias=bias)
        check(out, sums(torch.from_numpy(q).cuda(), b), torch.from_numpy(s).cuda(), scale, bias)


@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("m,n,k,pad", [(8, 1003, 14336, 0), (40, 515, 11008, 0), (300, 700, 28672, 8), (130, 513, 8200, 0), (7, 300, 10001, 1), (20, 300, 65536, 0)])
def test_linear_of_depths_past_8192(ops, dtype, m, n, k, pad):
    dtype = FLOATS[dtype]
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n)
    x = strided(m, k, dtype, pad)
    x.copy_(torch.randn(m, k, generator=g, device="cuda") * torch.exp(torch.randn(m, 1, generator=g, device="cuda")))
    x[2] = 0
    w, scale, bias = integers(k, n, k), torch.rand(n, generator=g, device="cuda") * 0.01, torch.randn(n, generator=g, device="cuda")
    out, two = (torch.empty(m, n, dtype=dtype, device="cuda") for _ in range(2))
    ops.linear_i8_dev(x, w, scale, out, bias=bias)
    q, s = ref.quantize(x.float().cpu().numpy())
    check(out, sums(torch.from_numpy(q).cuda(), w), torch.from_numpy(s).cuda(), scale, bias)
    dq, ds = strided(m, k, torch.int8, -k % 16), torch.empty(m, device="cuda")
    ops.quantize_rows_i8_dev(x, dq, ds)
    ops.matmul_i8_dev(dq, ds, w, scale, two, bias=bias)
    assert torch.equal(out, two)


# Tiles whose stages several CTA pairs share, for each width of a tile; n ends inside 16 bytes of a 16-bit row.
@pytest.mark.parametrize("m,n,k", [(20, 513, 8192), (50, 515, 8192), (100, 1001, 16384), (300, 517, 8192), (512, 7677, 24000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("room", [0, 3, 8])
def test_shared_tiles_that_end_inside_16_bytes(ops, m, n, k, dtype, room):
    a, b = integers(m, m, k), integers(n, n, k)
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    sa, sb, bias = torch.rand(m, generator=g, device="cuda") * 1e-5, torch.rand(n, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda")
    # room 8: rows on 16-byte boundaries, which tensor stores take; 0 and 3: rows off them
    pitch = -(-n // 8) * 8 + 8 if room == 8 else n + room
    whole = torch.full((m, pitch), 5.0, dtype=dtype, device="cuda")
    ops.matmul_i8_dev(a, sa, b, sb, whole[:, :n], bias=bias)
    check(whole[:, :n], sums(a, b), sa, sb, bias)
    assert bool((whole[:, n:] == 5).all())


SPECIAL = {"bf16": (2.0 ** -133, 3.0e38), "f16": (2.0 ** -24, 65504.0), "f32": (2.0 ** -149, 3.4e38)}


@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("cols,pad", [(300, 4), (300, 1), (1024, 0), (3000, 0), (3000, 1), (8192, 0), (9000, 0)])
def test_special_rows_of_every_type(ops, dtype, cols, pad):
    """Zeros, NaN, infinities, the type's smallest and largest values, in each of the quantising kernels; what a linear
    layer makes of them is what the two calls make."""
    tiny, large = SPECIAL[dtype]
    g = np.random.default_rng(cols)
    x = g.standard_normal((9, cols)).astype(np.float32)
    x[0] = 0
    x[1, 7] = np.nan
    x[2, cols - 1] = -np.inf
    x[3] = 0
    x[3, 5], x[3, 6] = tiny, -tiny
    x[4] = tiny * np.round(20 * g.standard_normal(cols))
    x[5] *= np.float32(large / 8)
    x[5, 0] = -large
    x[6, cols // 2], x[6, 0] = np.inf, np.nan
    x[7] = -0.0
    x = np.clip(x, -large, large, where=np.isfinite(x), out=x)
    dx = on_gpu(x, FLOATS[dtype], pad)
    q, s = run_quantize(ops, dx, -cols % 16)
    want_q, want_s = ref.quantize(dx.float().cpu().numpy())
    assert np.array_equal(q, want_q) and np.array_equal(s, want_s, equal_nan=True)
    w = integers(cols, 40, cols)
    one, two = (torch.empty(9, 40, device="cuda") for _ in range(2))
    ops.linear_i8_dev(dx, w, None, one)
    ops.matmul_i8_dev(on_gpu(q, None, -cols % 16), torch.from_numpy(s).cuda(), w, None, two)
    assert torch.equal(one.nan_to_num(nan=12345.0), two.nan_to_num(nan=12345.0))
    assert one.isnan().all(1).tolist() == np.isnan(want_s).tolist() and one.isnan().any(1).tolist() == np.isnan(want_s).tolist()


# Longer than the shared memory of sixteen CTAs: read again from L2.
LONG = [("f32", 600011), ("bf16", 900001), ("f16", 1100000)]


@pytest.mark.parametrize("dtype,vocab", LONG)
def test_long_rows_of_equal_scores(ops, dtype, vocab):
    g = np.random.default_rng(vocab)
    x = np.where(g.random((3, vocab)) < 0.3, g.integers(-3, 3, (3, vocab)), -1).astype(np.float32)
    x[1, ::7] = -np.inf
    x[2, ::5] = np.nan
    x = on_gpu(x, FLOATS[dtype], pad=3, offset=1)
    u = g.random(3).astype(np.float32)
    check_exact(ops, x, u)
    check_exact(ops, x, u, top_k=[vocab // 2, 5000, 2])
    check_exact(ops, x, u, top_p=np.array([0.5, 0.9, 0.01], np.float32))
    check_exact(ops, x, u, top_k=[vocab // 2, 300, 200000], top_p=np.array([0.99, 0.7, 0.9], np.float32), min_p=np.float32(0.01))


@pytest.mark.parametrize("dtype,vocab", LONG)
@pytest.mark.parametrize("spread", [0.01, 2.0, 6.0])
def test_long_rows_against_64_bits(ops, dtype, vocab, spread):
    g = np.random.default_rng(vocab + 1)
    x = (spread * g.standard_normal((3, vocab))).astype(np.float32)
    x[0] = np.sort(x[0])
    x[1, : vocab // 2] = -np.inf
    x = on_gpu(x, FLOATS[dtype])
    u = g.random(3).astype(np.float32)
    check_allowed(ops, x, u, min_p=[0.5, 0.01, 0.001])
    check_allowed(ops, x, u, temperature=0.7, top_k=[50, 3000, 9000])
    check_allowed(ops, x, u, temperature=0.7, top_p=np.array([0.3, 0.9, 0.99], np.float32))
    check_allowed(ops, x, u, temperature=0.7, top_k=[40, 2000, 30000], top_p=np.array([0.9, 0.95, 0.7], np.float32), min_p=0.01)


@pytest.mark.parametrize("dtype,vocab", [("f32", 300), ("bf16", 40000)] + LONG)
def test_greedy_and_masked_rows_of_every_length(ops, dtype, vocab):
    """Each row asks for something else; two have nothing to draw from."""
    g = np.random.default_rng(vocab)
    x = g.integers(-9, 9, (6, vocab)).astype(np.float32)
    x[1] = -np.inf
    x[4] = np.nan
    x[2, : vocab - 1] = -np.inf
    x[5, vocab // 2:] = np.inf
    x = on_gpu(x, FLOATS[dtype])
    token, logprob = run_sample(ops, x, 0.5, temperature=[0.0, 1.0, 1.0, -1.0, 0.0, 0.0], top_k=[0, 5, 9, 3, 1, 7],
                                top_p=[0.5, 0.9, 0.9, 0.1, 1.0, 1.0])
    best = [ref.sample_exact(row, 0.0, top_k=1)[0] for row in x.double().cpu().numpy()]
    assert token.tolist() == best and best[1] == best[4] == -1 and best[5] == vocab // 2
    assert logprob[[0, 2, 3, 5]].tolist() == [0.0] * 4 and np.isneginf(logprob[[1, 4]]).all()
