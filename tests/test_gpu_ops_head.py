"""The operators together, as a scoring head uses them; several handles at once; offsets past 32 bits."""
import numpy as np
import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


def test_scoring_head_draws_what_its_scores_allow():
    from examples.scoring_head import ScoringHead
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    rows = torch.randn(3001, 200, generator=g, device="cuda", dtype=torch.bfloat16)
    head = ScoringHead(rows, 40)
    q, s = ref.quantize(rows.float().cpu().numpy())
    assert np.array_equal(head.weights.cpu().numpy(), q) and np.array_equal(head.scale.cpu().numpy(), s)
    for b in (1, 3, 40):
        x = torch.randn(b, 200, generator=g, device="cuda", dtype=torch.bfloat16) * 0.3
        u = torch.rand(b, generator=g, device="cuda")
        k = torch.full((b,), 40, dtype=torch.int32, device="cuda")
        index, _ = head.draw(x, u, top_k=k, top_p=torch.full((b,), 0.9, device="cuda"))
        xq, xs = ref.quantize(x.float().cpu().numpy())
        exact = ref.product_sums(xq, q) * (xs.astype(np.float64)[:, None] * s.astype(np.float64))
        scores = head.scores[:b].double().cpu().numpy()
        assert (np.abs(scores - exact) <= 2.0 ** -8 * np.abs(exact) + 1e-30).all()
        for i in range(b):
            assert int(index[i]) in ref.sample_allowed(scores[i], float(u[i]), top_k=40, top_p=float(np.float32(0.9)))


def test_example_runs_and_repeats():
    from examples import scoring_head
    args = ["--rows", "5000", "--depth", "256", "--batch", "8", "--steps", "5"]
    first = scoring_head.main(args)
    assert len(first) == 6 and all(0 <= t < 5000 for step in first for t in step)
    assert scoring_head.main(args) == first


def test_two_handles_on_two_streams():
    """Each handle has its own workspace: calls on two streams may overlap."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    g = np.random.default_rng(5)
    work = []
    for s, (m, n, k) in zip(streams, [(300, 1000, 2048), (40, 4000, 1024)]):
        x = torch.from_numpy(g.standard_normal((m, k)).astype(np.float32)).cuda()
        w = torch.from_numpy(g.integers(-128, 128, (n, k), dtype=np.int8)).cuda()
        work.append((rbf.Ops(m, k, stream=s), x, w, torch.empty(m, n, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for o, x, w, out in work:
            o.linear_i8_dev(x, w, None, out)
    torch.cuda.synchronize()
    for o, x, w, out in work:
        q, s = ref.quantize(x.cpu().numpy())
        want = ref.product_sums(q, w.cpu().numpy()) * s.astype(np.float64)[:, None]
        # the sum's conversion and one product, half a unit of the last place each
        assert (np.abs(out.double().cpu().numpy() - want) <= 3 * 2.0 ** -24 * np.abs(want)).all()
        assert o.check_device_error() == rbf.RBF_OK
        o.close()


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart, in every matrix argument."""
    stride = (1 << 31) + 48
    big = torch.zeros(2 * stride + 4096, dtype=torch.int8, device="cuda")
    g = np.random.default_rng(6)
    a, b = g.integers(-128, 128, (5, 300), dtype=np.int8), g.integers(-128, 128, (3, 300), dtype=np.int8)
    far = torch.as_strided(big, (3, 300), (stride, 1))
    far.copy_(torch.from_numpy(b))
    with rbf.Ops(8, 4096, stream=torch.cuda.current_stream()) as o:
        for m in (2, 5):  # the kernel for few tokens, and the tensor cores'
            out = torch.empty(m, 3, dtype=torch.int32, device="cuda")
            o.matmul_i8_dev(torch.from_numpy(a[:m]).cuda(), None, far, None, out)
            assert np.array_equal(out.cpu().numpy(), ref.product_sums(a[:m], b))
            # and as the first operand
            out = torch.empty(3, m, dtype=torch.int32, device="cuda")
            o.matmul_i8_dev(far, None, torch.from_numpy(a[:m]).cuda(), None, out)
            assert np.array_equal(out.cpu().numpy(), ref.product_sums(b, a[:m]))
        far_out = torch.as_strided(big.view(torch.float32), (2, 8), (1 << 30, 1))
        o.matmul_i8_dev(torch.from_numpy(a[:2]).cuda(), None, torch.from_numpy(np.tile(b, (3, 1))[:8]).cuda(), None, far_out)
        assert np.array_equal(far_out.cpu().numpy(), ref.product_sums(a[:2], np.tile(b, (3, 1))[:8]).astype(np.float32))
        logits = torch.as_strided(big.view(torch.bfloat16), (2, 1000), ((1 << 30) + 8, 1))
        x = g.integers(-20, 3, (2, 1000)).astype(np.float32)
        logits.copy_(torch.from_numpy(x))
        u = np.array([0.3, 0.8], np.float32)
        token = torch.empty(2, dtype=torch.int32, device="cuda")
        o.sample_dev(logits, torch.from_numpy(u).cuda(), token, temperature=torch.full((2,), float(ref.LOG2E), device="cuda"))
        assert token.tolist() == [ref.sample_exact(x[i], float(u[i]))[0] for i in range(2)]
        q, s = torch.empty(2, 1000, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
        o.quantize_rows_i8_dev(logits, q, s)
        want_q, want_s = ref.quantize(x)
        assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)


@pytest.mark.parametrize("m,n,k", [(20, 300, 256), (100, 513, 512), (150, 777, 1500), (600, 1111, 640), (6000, 4001, 128)])
@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
def test_aligned_padded_outputs(name, m, n, k):
    """Output rows on 16-byte boundaries (stored by tensor copies) with padding behind them that stays as it was."""
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]
    g = np.random.default_rng(m)
    a, b = g.integers(-128, 128, (m, k), dtype=np.int8), g.integers(-128, 128, (n, k), dtype=np.int8)
    sa, sb = g.random(m).astype(np.float32) * 2.0 ** -12, g.random(n).astype(np.float32)
    whole = torch.full((m + 1, -(-n // 8) * 8 + 8), 5.0, dtype=dtype, device="cuda")
    with rbf.Ops(m, k, stream=torch.cuda.current_stream()) as o:
        o.matmul_i8_dev(torch.from_numpy(a).cuda(), torch.from_numpy(sa).cuda(), torch.from_numpy(b).cuda(), torch.from_numpy(sb).cuda(), whole[:m, :n])
        assert o.check_device_error() == rbf.RBF_OK
    want = ref.product_sums(a, b) * (sa.astype(np.float64)[:, None] * sb.astype(np.float64))
    off = np.abs(whole[:m, :n].double().cpu().numpy() - want)
    unit = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}[name]  # the last rounding, on top of three in fp32
    assert (off <= (unit + 4 * 2.0 ** -24) * np.abs(want) + (2.0 ** -25 if name == "f16" else 0)).all()
    assert bool((whole[:m, n:] == 5).all()) and bool((whole[m] == 5).all())


def test_a_product_may_take_longer_than_a_wait():
    """The bound on device-side waits is one on a step of the kernel: a product that takes several times as long is no
    timeout, and its result is the one that the kernel for few tokens gives."""
    m, n, k, bound = 4096, 131072, 32768, 4_000_000
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    a = torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    scale = torch.rand(m, generator=g, device="cuda") * 1e-4
    out, few = torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), torch.empty(2, n, dtype=torch.bfloat16, device="cuda")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with rbf.Ops(m, k, stream=torch.cuda.current_stream()) as o:
        for bad in (0, -1, 999_999):
            with pytest.raises(rbf.RbfError):
                o.set_timeout(bad)
        o.set_timeout(bound)
        o.matmul_i8_dev(a[:64], scale[:64], b[:1000], None, out[:64, :1000])  # loads the kernels
        begin.record()
        o.matmul_i8_dev(a, scale, b, None, out)
        end.record()
        assert o.check_device_error() == rbf.RBF_OK
        assert begin.elapsed_time(end) * 1e6 > 2 * bound  # else the bound was not passed
        for i in (0, m - 2):
            o.matmul_i8_dev(a[i:i + 2], scale[i:i + 2], b, None, few)
            assert torch.equal(out[i:i + 2], few)
