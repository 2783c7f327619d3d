"""The scoring-head operators against plain implementations in whole numbers
and 64 bits: 8-bit quantisation, the 8-bit product, the linear layer, sampling."""
import math

import numpy as np
import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu

FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# One rounding to the output's type, half a unit of its last place; fp32 results have three roundings (the sum's
# conversion, two scales) and the bias one more.
ROUNDING = {torch.float32: 4 * 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(4096, 8192, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == rbf.RBF_OK


def strided(rows, cols, dtype, pad, offset=0):
    """An empty [rows, cols] CUDA tensor in rows of cols + pad values, the first `offset` values into its memory."""
    return torch.empty(rows * (cols + pad) + offset + 1, dtype=dtype, device="cuda")[offset:offset + rows * (cols + pad)].view(
        rows, cols + pad)[:, :cols]


def on_gpu(values, dtype=None, pad=0, offset=0):
    t = torch.as_tensor(values)
    out = strided(t.shape[0], t.shape[1], dtype or t.dtype, pad, offset)
    out.copy_(t)
    return out


# ------------------------------------------------------------------ quantise

def run_quantize(ops, x, pad=0, offset=0):
    q = strided(*x.shape, torch.int8, pad, offset)
    q.fill_(77)
    s = torch.full((x.shape[0],), 7.0, device="cuda")
    ops.quantize_rows_i8_dev(x, q, s)
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (3, 7, 0, 0), (5, 128, 8, 0), (2, 1000, 0, 1), (9, 1024, 0, 0),
                                                  (4, 4096, 3, 5), (3, 8191, 1, 0), (2, 20001, 0, 0), (301, 64, 0, 0), (1, 65536, 0, 0)])
def test_quantize_equals_the_formula(ops, dtype, rows, cols, pad, offset):
    g = np.random.default_rng(rows * 1000 + cols)
    x = on_gpu((g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1)))).astype(np.float32), FLOATS[dtype], pad, offset)
    q, s = run_quantize(ops, x, pad, offset)
    want_q, want_s = ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(q, want_q) and np.array_equal(s, want_s)
    # And what it is for, in 64 bits: half a step off at most, and the rounding of 127 / t and of the product.
    x64, s64 = x.double().cpu().numpy(), s.astype(np.float64)[:, None]
    assert (np.abs(q * s64 - x64) <= s64 * (0.5 + 127 * 4 * 2.0 ** -24)).all()


def test_quantize_special_rows(ops):
    x = np.zeros((8, 300), np.float32)
    x[1, 7] = np.nan
    x[2, 299] = -np.inf
    x[3, 5], x[3, 6] = 2.0 ** -140, -(2.0 ** -142)     # subnormal
    x[4] = np.float32(3.0e38)
    x[5, 0] = -0.0
    x[6] = np.linspace(-1, 1, 300)
    x[7, 3] = 1.5 * 2.0 ** -101                         # 127 / t would overflow below 2^-120
    q, s = run_quantize(ops, on_gpu(x))
    want_q, want_s = ref.quantize(x)
    assert np.array_equal(q, want_q) and np.array_equal(s, want_s, equal_nan=True)


def test_quantize_halves_go_to_even(ops):
    x = np.concatenate([[127.0], np.arange(-126.5, 127, 1.0)]).astype(np.float32)[None]
    q, s = run_quantize(ops, on_gpu(x))
    assert s[0] == 1 and np.array_equal(q[0], np.rint(x[0]).astype(np.int8))


# ------------------------------------------------------------------- product

def i8(g, rows, cols):
    return g.integers(-128, 128, (rows, cols), dtype=np.int8)


def check_product(ops, a, b, pad_a=0, pad_b=0, off_b=0, pad_out=0, dtypes=("i32", "f32", "bf16", "f16"), seed=0):
    """Every output type of one product against the exact sums; the padding of the output stays as it was."""
    g = np.random.default_rng(seed)
    (m, k), n = a.shape, b.shape[0]
    da, db = on_gpu(a, None, pad_a), on_gpu(b, None, pad_b, off_b)
    sums = ref.product_sums(a, b)
    sa, sb = (np.exp(g.standard_normal(r)).astype(np.float32) * np.float32(2.0 ** -10) for r in (m, n))
    bias = g.standard_normal(n).astype(np.float32)
    for name in dtypes:
        dtype = torch.int32 if name == "i32" else FLOATS[name]
        whole = torch.full((m, n + pad_out), 3, dtype=dtype, device="cuda")
        out = whole[:, :n]
        if name == "i32":
            ops.matmul_i8_dev(da, None, db, None, out)
            assert np.array_equal(out.cpu().numpy(), sums), (m, n, k)
        else:
            for with_bias in (False, True):
                ops.matmul_i8_dev(da, torch.from_numpy(sa).cuda(), db, torch.from_numpy(sb).cuda(), out,
                                  bias=torch.from_numpy(bias).cuda() if with_bias else None)
                scaled = sums * (sa.astype(np.float64)[:, None] * sb.astype(np.float64))
                want = scaled + (bias.astype(np.float64) if with_bias else 0.0)
                off = np.abs(out.double().cpu().numpy() - want)
                room = ROUNDING[dtype] * np.abs(want) + 4 * 2.0 ** -24 * (np.abs(scaled) + np.abs(want)) + (2.0 ** -25 if name == "f16" else 0)
                assert (off <= room).all(), (name, m, n, k, off.max())
        if pad_out:
            assert bool((whole[:, n:] == 3).all())


SIZES = [(1, 1, 1), (1, 1, 16), (1, 300, 64), (2, 257, 128), (3, 130, 100), (5, 1000, 384), (16, 512, 129), (17, 4097, 768), (33, 255, 1000),
         (64, 256, 1024), (65, 700, 1040), (100, 129, 2048), (129, 384, 260), (256, 513, 768), (257, 640, 1152), (300, 1025, 333), (513, 256, 2500)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_is_exact(ops, m, n, k):
    g = np.random.default_rng(m + 31 * n + 7 * k)
    check_product(ops, i8(g, m, k), i8(g, n, k), pad_a=-k % 16, pad_b=-k % 16, pad_out=3)


@pytest.mark.parametrize("pad_a,pad_b,off_b", [(0, 0, 0), (1, 3, 0), (0, 4, 4), (5, 8, 1), (7, 13, 16), (0, 13, 3)])
@pytest.mark.parametrize("m,n,k", [(1, 70, 99), (40, 200, 203)])
def test_product_of_any_stride_and_alignment(ops, m, n, k, pad_a, pad_b, off_b):
    g = np.random.default_rng(m + pad_a * 100 + pad_b)
    check_product(ops, i8(g, m, k), i8(g, n, k), pad_a, pad_b, off_b)


@pytest.mark.parametrize("m,n,k", [(1, 200, 8192), (40, 300, 8192), (200, 300, 4100), (300, 257, 8192)])
def test_sums_past_24_bits_stay_exact(ops, m, n, k):
    """Rows of equal extreme values: the sums pass 2^24, where an fp32 running sum would lose their last bits."""
    g = np.random.default_rng(k)
    a = np.where(g.random((m, k)) < 0.97, 127, 126).astype(np.int8)
    b = np.where(g.random((n, k)) < 0.97, 127, 125).astype(np.int8)
    a[0], b[0] = -128, -128
    check_product(ops, a, b, pad_a=-k % 16, pad_b=-k % 16, dtypes=("i32", "f32"))


@pytest.mark.parametrize("m,n,k", [(4, 40000, 512), (128, 20011, 384), (4096, 300, 64), (1500, 1300, 700), (4, 256, 8192), (32, 1024, 8192)])
def test_many_tiles_and_few(ops, m, n, k):
    g = np.random.default_rng(m * n)
    check_product(ops, i8(g, m, k), i8(g, n, k), pad_a=-k % 16, pad_b=-k % 16, dtypes=("i32", "bf16"))


def test_calls_on_one_handle_do_not_meet(ops):
    """Different shapes back to back on the handle's workspace, without a wait between them."""
    g = np.random.default_rng(9)
    calls = []
    for m, n, k in [(300, 700, 1000), (1, 5000, 256), (40, 300, 4096), (256, 256, 64), (7, 90, 8000)] * 3:
        a, b = i8(g, m, k), i8(g, n, k)
        calls.append((a, b, on_gpu(a, None, -k % 16), on_gpu(b, None, -k % 16), torch.empty(m, n, dtype=torch.int32, device="cuda")))
    for _, _, da, db, out in calls:
        ops.matmul_i8_dev(da, None, db, None, out)
    for a, b, _, _, out in calls:
        assert np.array_equal(out.cpu().numpy(), ref.product_sums(a, b))


def test_depth_zero_and_empty(ops):
    bias = torch.arange(5, dtype=torch.float32, device="cuda")
    out = torch.full((3, 5), 9.0, device="cuda")
    empty = lambda r: torch.empty(r, 0, dtype=torch.int8, device="cuda")  # noqa: E731
    ops.matmul_i8_dev(empty(3), None, empty(5), None, out, bias=bias)
    assert bool((out == bias).all())
    ops.matmul_i8_dev(empty(3), None, empty(5), None, out)
    assert bool((out == 0).all())
    ops.matmul_i8_dev(empty(0), None, empty(5), None, torch.empty(0, 5, device="cuda"))
    ops.matmul_i8_dev(empty(3), None, empty(0), None, torch.empty(3, 0, device="cuda"))
    assert ops.last_launches == 0


def test_scale_specials_reach_the_result(ops):
    """A NaN scale (of a row that held a NaN) makes its row NaN and no other; an infinite bias stays."""
    a, b = on_gpu(np.full((3, 64), 2, np.int8)), on_gpu(np.full((4, 64), 3, np.int8))
    sa = torch.tensor([1.0, math.nan, 1.0], device="cuda")
    bias = torch.tensor([0.0, math.inf, 0.0, 1.0], device="cuda")
    out = torch.empty(3, 4, device="cuda")
    ops.matmul_i8_dev(a, sa, b, None, out, bias=bias)
    assert bool(out[1].isnan().all()) and out[0].tolist() == [384.0, math.inf, 384.0, 385.0]


# -------------------------------------------------------------------- linear

@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("m,n,k,pad", [(1, 50, 64, 0), (1, 1000, 768, 0), (3, 700, 1000, 8), (31, 300, 2049, 1), (130, 260, 4096, 0), (300, 520, 384, 0)])
def test_linear_is_quantize_then_product(ops, dtype, m, n, k, pad):
    g = np.random.default_rng(m + n + k)
    x = on_gpu(g.standard_normal((m, k)).astype(np.float32), FLOATS[dtype], pad)
    if m > 2:
        x[1] = 0
    w, sw = on_gpu(i8(g, n, k), None, -k % 16), torch.rand(n, device="cuda") * 0.01
    bias = torch.randn(n, device="cuda")
    out = torch.empty(m, n, dtype=FLOATS[dtype], device="cuda")
    ops.linear_i8_dev(x, w, sw, out, bias=bias)
    q, s = ref.quantize(x.float().cpu().numpy())
    scaled = ref.product_sums(q, w.cpu().numpy()) * (s.astype(np.float64)[:, None] * sw.double().cpu().numpy())
    want = scaled + bias.double().cpu().numpy()
    off = np.abs(out.double().cpu().numpy() - want)
    assert (off <= ROUNDING[FLOATS[dtype]] * np.abs(want) + 4 * 2.0 ** -24 * (np.abs(scaled) + np.abs(want)) + 2.0 ** -25).all()
    # The same call in its two steps gives the same bits.
    dq, ds = strided(m, k, torch.int8, -k % 16), torch.empty(m, device="cuda")
    ops.quantize_rows_i8_dev(x, dq, ds)
    two = torch.empty_like(out)
    ops.matmul_i8_dev(dq, ds, w, sw, two, bias=bias)
    assert torch.equal(out, two)


def test_linear_rows_that_hold_nan(ops):
    x = torch.ones(3, 128, device="cuda")
    x[1, 5] = math.nan
    out = torch.empty(3, 40, device="cuda")
    ops.linear_i8_dev(x, torch.ones(40, 128, dtype=torch.int8, device="cuda"), None, out)
    assert bool(out[1].isnan().all()) and bool(out[[0, 2]].isfinite().all())


# ------------------------------------------------------------------ sampling

def run_sample(ops, x, u, **ask):
    rows = x.shape[0]
    vec = lambda v, t: torch.as_tensor(np.broadcast_to(np.asarray(v), (rows,)).copy()).to(t).cuda()  # noqa: E731
    token, logprob = torch.full((rows,), -7, dtype=torch.int32, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    kw = {k: vec(v, torch.int32 if k == "top_k" else torch.float32) for k, v in ask.items()}
    ops.sample_dev(x, vec(u, torch.float32), token, logprob, **kw)
    return token.cpu().numpy(), logprob.cpu().numpy()


LOGPROB_ROOM = 3e-6  # log of a quotient of exact whole numbers: three roundings and logf's one, relative, plus 2^-24 near zero


def check_exact(ops, x, u, **ask):
    """Whole-numbered scores at temperature log2(e): every weight is a power of two, and the result is one index."""
    token, logprob = run_sample(ops, x, u, temperature=ref.LOG2E, **ask)
    xs = x.double().cpu().numpy()
    at = lambda v, i: np.broadcast_to(np.asarray(v), (xs.shape[0],))[i].item()  # noqa: E731
    for i in range(xs.shape[0]):
        want, lp = ref.sample_exact(xs[i], at(u, i), **{k: at(v, i) for k, v in ask.items()})
        assert token[i] == want, (i, token[i], want, {k: at(v, i) for k, v in ask.items()}, at(u, i))
        assert logprob[i] == lp or abs(logprob[i] - lp) <= LOGPROB_ROOM * max(abs(lp), 2.0 ** -24), (i, logprob[i], lp)


VOCABS = [1, 2, 7, 31, 33, 255, 1000, 4097, 20011]


@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("vocab", VOCABS)
def test_sample_whole_numbers(ops, dtype, vocab):
    """Few different scores, so ties everywhere: plain, top-k, top-p, min-p and all of them, each from both ends of u."""
    g = np.random.default_rng(vocab)
    rows = 12
    x = g.integers(-30, 4, (rows, vocab)).astype(np.float32)
    x[1] = 2.0                                      # one single score
    x[2, g.random(vocab) < 0.9] = -np.inf           # mostly masked
    x[3] = -np.inf
    x[4, vocab // 2] = 40.0                         # all else is below 2^-36 of it
    x[5, g.random(vocab) < 0.3] = np.nan
    x[6] = np.where(g.random(vocab) < 0.5, 0.0, -0.0)
    x[7, 0] = np.inf
    x = on_gpu(x, FLOATS[dtype], pad=vocab % 3, offset=vocab % 2)
    u = g.random(rows).astype(np.float32)
    k = g.integers(1, vocab + 2, rows)
    p = g.random(rows).astype(np.float32)
    mp = (g.random(rows) ** 3).astype(np.float32)
    for uu in (u, 0.0, np.float32(1 - 2.0 ** -24)):
        check_exact(ops, x, uu)
        check_exact(ops, x, uu, top_k=k)
        check_exact(ops, x, uu, top_k=1 + k % 3)
        check_exact(ops, x, uu, top_p=p)
        check_exact(ops, x, uu, min_p=mp)
        check_exact(ops, x, uu, top_k=k, top_p=p, min_p=mp)


@pytest.mark.parametrize("vocab", [3, 1500, 30000])
def test_sample_parameter_edges(ops, vocab):
    g = np.random.default_rng(vocab)
    x = on_gpu(g.integers(-12, 4, (6, vocab)).astype(np.float32))
    u = g.random(6).astype(np.float32)
    check_exact(ops, x, u, top_k=[0, -5, vocab, vocab + 1, 1, 2])
    check_exact(ops, x, u, top_p=[0.0, -1.0, 1.0, 5.0, 1e-9, 0.999])
    check_exact(ops, x, u, min_p=[0.0, -1.0, 1.0, 2.0, 1e-12, 0.5])
    check_exact(ops, x, [0.0, -1.0, 1.0, 2.0, 0.999, 1e-9])
    nan = float("nan")
    plain, _ = run_sample(ops, x, u)
    same, _ = run_sample(ops, x, u, top_p=nan, min_p=nan)
    assert np.array_equal(plain, same)
    assert np.array_equal(run_sample(ops, x, nan)[0], run_sample(ops, x, 0.0)[0])
    best = np.argmax(x.cpu().numpy(), 1)
    for t in (0.0, -1.0, nan, -math.inf):
        token, logprob = run_sample(ops, x, u, temperature=t)
        assert np.array_equal(token, best) and (logprob == 0).all()


def check_allowed(ops, x, u, **ask):
    token, logprob = run_sample(ops, x, u, **ask)
    xs = x.double().cpu().numpy()
    at = lambda v, i: np.broadcast_to(np.asarray(v), (xs.shape[0],))[i].item()  # noqa: E731
    for i in range(xs.shape[0]):
        allowed = ref.sample_allowed(xs[i], at(u, i), **{k: at(v, i) for k, v in ask.items()})
        assert int(token[i]) in allowed, (i, token[i], allowed)
        assert any(logprob[i] == lp or abs(logprob[i] - lp) <= 2 * ref.WEIGHT_ERROR * max(1.0, abs(lp)) for lp in allowed[int(token[i])]), (
            i, logprob[i], allowed[int(token[i])])


@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("vocab,spread", [(50, 1.0), (1000, 3.0), (5000, 0.01), (32000, 2.5), (32003, 0.0), (128000, 1.0), (150001, 6.0)])
def test_sample_against_64_bits(ops, dtype, vocab, spread):
    g = np.random.default_rng(vocab)
    rows = 6
    x = (spread * g.standard_normal((rows, vocab))).astype(np.float32)
    x[0, : vocab // 2] = -np.inf
    x[1, g.integers(0, vocab, 5)] += 9
    x = on_gpu(x, FLOATS[dtype])
    u = g.random(rows).astype(np.float32)
    t = (0.3 + g.random(rows)).astype(np.float32)
    check_allowed(ops, x, u)
    check_allowed(ops, x, u, temperature=t, top_k=[1, 5, 50, 300, 3000, vocab - 1])
    check_allowed(ops, x, u, temperature=t, top_p=[0.1, 0.5, 0.9, 0.95, 0.99, 0.999])
    check_allowed(ops, x, u, temperature=t, min_p=[0.5, 0.1, 0.05, 0.01, 0.001, 0.9])
    check_allowed(ops, x, u, temperature=t, top_k=[40, 2000, vocab, 10, 700, 1500], top_p=[0.9, 0.8, 0.99, 0.3, 0.95, 0.7], min_p=0.01)


@pytest.mark.parametrize("rows,vocab", [(1, 1000003), (2, 400000), (300, 700), (700, 33)])
def test_sample_long_rows_and_many(ops, rows, vocab):
    g = np.random.default_rng(rows)
    x = on_gpu((3 * g.standard_normal((rows, vocab))).astype(np.float32))
    u = g.random(rows).astype(np.float32)
    check_allowed(ops, x, u)
    check_allowed(ops, x, u, top_k=20, top_p=np.float32(0.9))
    check_allowed(ops, x, u, top_p=np.float32(0.95))


def test_sample_infinite_temperature_and_mask(ops):
    """At infinite temperature every score that is not masked is as likely as any other."""
    x = torch.randn(1, 1000, device="cuda")
    x[0, 100:] = -math.inf
    for u in (0.0, 0.255, 0.9999):
        token, logprob = run_sample(ops, x, u, temperature=math.inf)
        assert token[0] == int(u * 100) and abs(logprob[0] + math.log(100)) < 1e-5
    x[0, 100:] = torch.finfo(torch.float32).min  # a mask of the type's lowest value is a score like any other
    token, _ = run_sample(ops, x, 0.9999, temperature=1.0)
    assert token[0] < 100


def test_sample_rows_do_not_meet(ops):
    """A row's result depends on that row alone."""
    x = torch.randn(64, 5000, device="cuda") * 3
    u = torch.rand(64).numpy()
    token, logprob = run_sample(ops, x, u, top_p=np.float32(0.9))
    for i in (0, 17, 63):
        t, lp = run_sample(ops, x[i:i + 1].contiguous(), u[i:i + 1], top_p=np.float32(0.9))
        assert t[0] == token[i] and lp[0] == logprob[i]


def test_sample_without_columns_or_logprob(ops):
    token, logprob = run_sample(ops, torch.empty(3, 0, device="cuda"), 0.5)
    assert token.tolist() == [-1] * 3 and np.isneginf(logprob).all()
    x = torch.randn(4, 100, device="cuda")
    t = torch.empty(4, dtype=torch.int32, device="cuda")
    ops.sample_dev(x, torch.full((4,), 0.5, device="cuda"), t)
    assert t.tolist() == run_sample(ops, x, 0.5)[0].tolist()


def test_sample_frequencies(ops):
    """20,000 draws from eight scores: each count within 5 standard deviations."""
    x = torch.tensor([0.0, 1.0, 2.0, -1.0, 0.5, -math.inf, 1.5, 0.0], device="cuda")
    n = 20000
    token, _ = run_sample(ops, x.expand(n, 8).contiguous(), np.random.default_rng(4).random(n).astype(np.float32))
    p = torch.softmax(x.double(), 0).cpu().numpy()
    count = np.bincount(token, minlength=8)
    assert (np.abs(count - n * p) <= 5 * np.sqrt(n * p * (1 - p))).all()


# ---------------------------------------------------- the handle, and refusals

def test_launch_failures_are_reported(ops):
    x, out = torch.ones(2, 64, device="cuda"), torch.zeros(2, 8, device="cuda")
    w = torch.ones(8, 64, dtype=torch.int8, device="cuda")
    ops.inject_host_fault(1)
    with pytest.raises(rbf.RbfError) as e:
        ops.linear_i8_dev(x, w, None, out)
    assert e.value.status == rbf.RBF_ERR_CUDA
    ops.linear_i8_dev(x, w, None, out)
    # 64 products of 127 * 1, times the scale 1 / 127, in fp32
    assert bool((out - 64.0).abs().max() <= 64 * 4 * 2.0 ** -24) and ops.check_device_error() == rbf.RBF_OK


def test_own_stream():
    with rbf.Ops(8, 256) as o:
        x = torch.randn(8, 1000, device="cuda")
        u, t = torch.rand(8, device="cuda"), torch.empty(8, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        o.sample_dev(x, u, t, top_k=torch.full((8,), 1, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(t.long(), x.argmax(1))


def test_c_entry_points_refuse_bad_arguments(ops):
    """Through the library itself: sizes, strides, alignment, types, missing pointers."""
    lib, h, bad = ops.lib, ops._h, rbf.RBF_ERR_INVALID_VALUE
    buf = torch.zeros(4096, device="cuda")
    p = buf.data_ptr()
    assert lib.quantize_rows_i8_dev(h, p, 0, 4, 2, 5, p + 1024, 5, p + 2048) == bad       # stride under the row
    assert lib.quantize_rows_i8_dev(h, p, 3, 5, 2, 5, p + 1024, 5, p + 2048) == bad       # an integer type
    assert lib.quantize_rows_i8_dev(h, p + 2, 0, 5, 2, 5, p + 1024, 5, p + 2048) == bad   # off its element's boundary
    assert lib.quantize_rows_i8_dev(h, p, 0, 5, -1, 5, p + 1024, 5, p + 2048) == bad
    assert lib.quantize_rows_i8_dev(h, None, 0, 5, 2, 5, p + 1024, 5, p + 2048) == bad
    assert lib.quantize_rows_i8_dev(h, p, 0, 5, 2, 5, p + 1024, 5, None) == bad
    assert lib.matmul_i8_dev(h, p, 8, None, p, 7, None, None, p + 1024, 0, 4, 2, 4, 8) == bad
    assert lib.matmul_i8_dev(h, p, 8, None, p, 8, None, None, p + 1024, 0, 3, 2, 4, 8) == bad
    assert lib.matmul_i8_dev(h, p, 8, None, p, 8, None, None, p + 1026, 0, 4, 2, 4, 8) == bad
    assert lib.matmul_i8_dev(h, p, 8, p, p, 8, None, None, p + 1024, 3, 4, 2, 4, 8) == bad  # scales on raw sums
    assert lib.matmul_i8_dev(h, p, 8, None, p, 8, None, None, p + 1024, 4, 4, 2, 4, 8) == bad
    assert lib.matmul_i8_dev(h, p, 8, None, None, 8, None, None, p + 1024, 0, 4, 2, 4, 8) == bad
    assert lib.linear_i8_dev(h, p, 0, 8, p, 8, None, None, p + 1024, 3, 4, 2, 4, 8) == bad
    assert lib.linear_i8_dev(h, p, 0, 7, p, 8, None, None, p + 1024, 0, 4, 2, 4, 8) == bad
    assert lib.sample_dev(h, p, 0, 8, 2, 9, p, None, None, None, None, p + 1024, None) == bad
    assert lib.sample_dev(h, p, 0, 8, 2, 8, None, None, None, None, None, p + 1024, None) == bad
    assert lib.sample_dev(h, p, 0, 8, 2, 8, p, None, None, None, None, None, None) == bad
    assert lib.sample_dev(h, p, 0, 1 << 27, 1, (1 << 26) + 1, p, None, None, None, None, p + 1024, None) == bad
    assert bool((buf == 0).all())


def test_handle_limits(ops):
    small = rbf.Ops(4, 64)
    w = torch.ones(8, 65, dtype=torch.int8, device="cuda")
    for bad in (lambda: small.matmul_i8_dev(torch.ones(5, 64, dtype=torch.int8, device="cuda"), None, w[:, :64], None, torch.empty(5, 8, device="cuda")),
                lambda: small.matmul_i8_dev(torch.ones(4, 65, dtype=torch.int8, device="cuda"), None, w, None, torch.empty(4, 8, device="cuda")),
                lambda: small.linear_i8_dev(torch.ones(5, 64, device="cuda"), w[:, :64], None, torch.empty(5, 8, device="cuda")),
                lambda: rbf.Ops(0, 64), lambda: rbf.Ops(1, 0), lambda: rbf.Ops(1, rbf.RBF_OPS_MAX_DEPTH + 1), lambda: rbf.Ops((1 << 20) + 1, 1)):
        with pytest.raises(rbf.RbfError) as e:
            bad()
        assert e.value.status == rbf.RBF_ERR_INVALID_VALUE
    small.close()


@pytest.mark.parametrize("dtype,vocab", [("bf16", 300000), ("f32", 70001)])
def test_sample_thousands_of_equal_scores(ops, dtype, vocab):
    """The kept prefix ends among thousands of equal scores, which no bins divide."""
    g = np.random.default_rng(vocab)
    x = on_gpu(np.where(g.random((4, vocab)) < 0.3, g.integers(-3, 3, (4, vocab)), -1).astype(np.float32), FLOATS[dtype])
    u = g.random(4).astype(np.float32)
    check_exact(ops, x, u, top_k=[vocab // 2, 5000, 2, vocab - 3])
    check_exact(ops, x, u, top_p=np.array([0.5, 0.9, 0.01, 0.99], np.float32))
    check_exact(ops, x, u, top_k=[vocab // 2, 5000, 300, vocab - 3], top_p=np.array([0.5, 0.9, 0.7, 0.99], np.float32))


@pytest.mark.parametrize("order", [1, -1])
def test_sample_sorted_rows(ops, order):
    """Sorted scores put all candidates into one part of the row."""
    x = torch.sort(3 * torch.randn(3, 50000, device="cuda"), dim=1, descending=order < 0)[0].contiguous()
    u = np.array([0.1, 0.5, 0.99], np.float32)
    check_allowed(ops, x, u, top_k=[3, 300, 4000])
    check_allowed(ops, x, u, top_p=np.array([0.5, 0.9, 0.99], np.float32))
    check_allowed(ops, x, u, top_k=[50, 300, 4000], top_p=np.array([0.5, 0.9, 0.99], np.float32), min_p=0.001)


@pytest.mark.parametrize("rows,vocab", [(3, 10000), (64, 10001), (300, 17000), (9, 150001), (4, 400000)])
def test_sample_clusters_beside_other_work(ops, rows, vocab):
    """Another stream's kernels come and go, so that the CTAs of a row's cluster find room at different times: every
    call has the row's one result (whole-numbered scores, whose weights are powers of two)."""
    g = np.random.default_rng(vocab)
    x = g.integers(-30, 4, (rows, vocab)).astype(np.float32)
    x[:, vocab // 3] = 9.0
    u = g.random(rows).astype(np.float32)
    want = [ref.sample_exact(x[i], float(u[i]), top_p=0.9)[0] for i in range(min(rows, 6))]
    dx, du = on_gpu(x), torch.from_numpy(u).cuda()
    t, p = torch.full((rows,), float(ref.LOG2E), device="cuda"), torch.full((rows,), 0.9, device="cuda")
    tokens = [torch.full((rows,), -7, dtype=torch.int32, device="cuda") for _ in range(40)]
    other, busy = torch.cuda.Stream(), torch.zeros(1 << 22, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(200):
            busy.add_(1.0)
    for token in tokens:
        ops.sample_dev(dx, du, token, temperature=t, top_p=p)
    torch.cuda.synchronize()
    assert tokens[0][:6].tolist() == want
    assert all(torch.equal(token, tokens[0]) for token in tokens)


def test_quantize_the_longest_row(ops):
    """2^31 - 1 columns, the most that a call takes: column numbers do not pass 32 bits at the row's end."""
    cols = (1 << 31) - 1
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.empty(1, cols, dtype=torch.bfloat16, device="cuda")
    for c in range(0, cols, 1 << 28):
        x[:, c:c + (1 << 28)] = torch.randn(1, min(1 << 28, cols - c), generator=g, device="cuda")
    x[0, -1] = 100.0  # the largest one is the last
    whole = torch.full((1, cols + 65), 77, dtype=torch.int8, device="cuda")
    scale = torch.empty(1, device="cuda")
    ops.quantize_rows_i8_dev(x, whole[:, :cols], scale)
    assert scale[0].item() == np.float32(100) * (np.float32(1) / np.float32(127))
    factor = float((np.float32(1) / np.float32(100)) * np.float32(127))
    for c in range(0, cols, 1 << 28):
        part = x[:, c:c + (1 << 28)].float()
        assert torch.equal(whole[:, c:min(c + (1 << 28), cols)], (part * factor).round_().to(torch.int8))
    assert bool((whole[:, cols:] == 77).all())


@pytest.mark.parametrize("temperature", [1e-45, 1e-39, 4e-39, 4.5e-39, 1e-30])
@pytest.mark.parametrize("vocab", [40, 5000, 300000])
def test_sample_temperatures_next_to_zero(ops, vocab, temperature):
    """Every temperature above 0 draws: so near to it among the scores that equal the best one."""
    g = np.random.default_rng(vocab)
    x = on_gpu(np.minimum(g.integers(-30, 6, (4, vocab)), 4).astype(np.float32))
    u = np.array([0.0, 0.3, 0.7, 0.999], np.float32)
    check_allowed(ops, x, u, temperature=temperature)
    check_allowed(ops, x, u, temperature=temperature, min_p=0.1)
    check_allowed(ops, x, u, temperature=temperature, top_k=[2, 7, 30, vocab - 1])
    check_allowed(ops, x, u, temperature=temperature, top_p=np.array([0.1, 0.5, 0.9, 0.99], np.float32))
    check_allowed(ops, x, u, temperature=temperature, top_k=[2, 7, 30, vocab - 1], top_p=np.float32(0.6), min_p=0.5)


@pytest.mark.parametrize("temperature", [1e38, 1.3e38, 3e38, math.inf])
def test_sample_temperatures_next_to_infinity(ops, temperature):
    """Finite scores as far apart as their type allows, among them masks of its lowest value: at infinite temperature
    all are alike. (Scores whose difference passes the largest float are infinitely far apart.)"""
    lowest = torch.finfo(torch.float32).min
    g = np.random.default_rng(3)
    x = g.standard_normal((3, 2000)).astype(np.float32)
    x[0, g.random(2000) < 0.5] = lowest
    x[1] *= np.float32(3e37)
    x[2] = np.where(g.random(2000) < 0.9, np.float32(lowest), np.float32(-1e38))
    x = on_gpu(x)
    for u in (0.0, 0.2, 0.61, 0.9999):
        check_allowed(ops, x, u, temperature=temperature)
        check_allowed(ops, x, u, temperature=temperature, top_p=np.float32(0.4))
        check_allowed(ops, x, u, temperature=temperature, min_p=0.3)
