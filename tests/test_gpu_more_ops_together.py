"""8-bit floating-point products, verification and distillation together, as a user has them: one after the other on one
stream, captured, on two handles at once, over long rows, after failed launches."""
import math

import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import more_ops_reference as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Head:
    """A head of `vocab` channels in 8-bit floating point (a scale for each 128 x 128), of a target and of a draft, and
    what a step of either of its two uses writes."""

    def __init__(self, ops, seqs, drafts, vocab, depth, seed):
        g = gen(seed)
        self.ops, self.seqs, self.drafts, self.vocab, self.depth = ops, seqs, drafts, vocab, depth
        rows = seqs * (drafts + 1)
        self.weights = torch.randn(vocab, depth, generator=g, device="cuda") * depth ** -0.5 * 2.0
        self.w8, self.w_scale = torch.empty(vocab, depth, dtype=E4M3, device="cuda"), torch.empty(-(-vocab // 128), -(-depth // 128), device="cuda")
        self.x = torch.randn(rows, depth, generator=g, device="cuda").bfloat16()
        self.near = (self.x.float().view(seqs, drafts + 1, depth)[:, :drafts] + 0.2 * torch.randn(seqs, drafts, depth, generator=g, device="cuda"))
        self.near = self.near.reshape(seqs * drafts, depth).bfloat16()
        self.u = torch.rand(seqs, drafts + 1, generator=g, device="cuda")
        self.u_draft = torch.rand(seqs * drafts, generator=g, device="cuda")
        blocks = -(-depth // 128)
        self.x8, self.x_scale = torch.empty(rows, depth, dtype=E4M3, device="cuda"), torch.empty(rows, blocks, device="cuda")
        self.near8, self.near_scale = torch.empty(seqs * drafts, depth, dtype=E4M3, device="cuda"), torch.empty(seqs * drafts, blocks, device="cuda")
        self.target = torch.empty(seqs, drafts + 1, vocab, dtype=torch.bfloat16, device="cuda")
        self.draft = torch.empty(seqs, drafts, vocab, dtype=torch.bfloat16, device="cuda")
        self.drafted = torch.empty(seqs, drafts, dtype=torch.int32, device="cuda")
        self.token = torch.empty(seqs, drafts + 1, dtype=torch.int32, device="cuda")
        self.accepted = torch.empty(seqs, dtype=torch.int32, device="cuda")
        self.logprob = torch.empty(seqs, drafts + 1, device="cuda")
        # training: the target's scores against a list of their best, a few places off
        self.index = torch.randint(0, vocab, (rows, 8), generator=g, device="cuda", dtype=torch.int32)
        self.teacher = torch.randn(rows, 8, generator=g, device="cuda") * 2
        self.loss, self.grad = torch.empty(rows, device="cuda"), torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
        self.grad8, self.grad_scale = torch.empty(rows, vocab, dtype=E5M2, device="cuda"), torch.empty(rows, -(-vocab // 128), device="cuda")
        self.wt8, self.wt_scale = torch.empty(depth, vocab, dtype=E4M3, device="cuda"), torch.empty(blocks, -(-vocab // 128), device="cuda")
        self.wt = self.weights.t().contiguous()
        self.dx = torch.empty(rows, depth, device="cuda")
        self.clear()
        torch.cuda.synchronize()

    def answer(self):
        """Weights and tokens to 8 bits, the target's scores and the draft's, its tokens, and their check."""
        o = self.ops
        o.quantize_f8_dev(self.weights, self.w8, self.w_scale, block_rows=128)
        o.quantize_f8_dev(self.x, self.x8, self.x_scale)
        o.quantize_f8_dev(self.near, self.near8, self.near_scale)
        o.matmul_f8_dev(self.x8, self.x_scale, self.w8, self.w_scale, self.target.view(-1, self.vocab))
        o.matmul_f8_dev(self.near8, self.near_scale, self.w8, self.w_scale, self.draft.view(-1, self.vocab))
        o.sample_dev(self.draft.view(-1, self.vocab), self.u_draft, self.drafted.view(-1))
        o.verify_dev(self.target, self.drafted, self.u, self.token, self.accepted, d_logprob=self.logprob, d_draft=self.draft)

    def learn(self):
        """The scores' loss and gradient, and that of the head's input."""
        o = self.ops
        o.quantize_f8_dev(self.weights, self.w8, self.w_scale, block_rows=128)
        o.quantize_f8_dev(self.wt, self.wt8, self.wt_scale, block_rows=128)
        o.quantize_f8_dev(self.x, self.x8, self.x_scale)
        o.matmul_f8_dev(self.x8, self.x_scale, self.w8, self.w_scale, self.target.view(-1, self.vocab))
        o.distill_dev(self.target.view(-1, self.vocab), self.index, self.teacher, d_loss=self.loss, d_grad=self.grad, temperature=2.0)
        o.quantize_f8_dev(self.grad, self.grad8, self.grad_scale)
        o.matmul_f8_dev(self.grad8, self.grad_scale, self.wt8, self.wt_scale, self.dx)

    def outputs(self):
        return [t.clone() for t in (self.w8.view(torch.uint8), self.x8.view(torch.uint8), self.target, self.draft, self.drafted, self.token,
                                    self.accepted, self.logprob, self.loss, self.grad, self.dx)]

    def clear(self):
        for t in (self.target, self.draft, self.drafted, self.token, self.accepted, self.logprob, self.loss, self.grad, self.dx):
            t.zero_()
        for t in (self.w8, self.x8, self.near8, self.grad8, self.wt8):
            t.view(torch.uint8).zero_()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def check_answer(h):
    """Each step against the definition, on what the step before it wrote."""
    for x, x8, scale, block_rows in ((h.weights, h.w8, h.w_scale, 128), (h.x, h.x8, h.x_scale, 1), (h.near, h.near8, h.near_scale, 1)):
        want, want_scale = ref.quantize_f8(x, E4M3, block_rows)
        assert torch.equal(x8.double(), want) and torch.equal(scale, want_scale)
    for x8, scale, out in ((h.x8, h.x_scale, h.target), (h.near8, h.near_scale, h.draft)):
        want, size = ref.product(x8, scale, h.w8, h.w_scale, 128)
        off = (out.view(-1, h.vocab).double() - want).abs()
        assert bool((off <= ref.product_error(size, h.depth, torch.bfloat16, want)).all())
    ref.check_verify(h.target.cpu(), h.draft.cpu(), h.drafted.cpu(), None, h.u.cpu(), None, h.token.cpu(), h.accepted.cpu(), h.logprob.cpu())


def test_draft_and_verify_through_a_quantised_head():
    with rbf.Ops(64, 512, stream=torch.cuda.current_stream()) as o:
        h = Head(o, 5, 4, 1003, 320, seed=1)
        h.answer()
        assert o.check_device_error() == rbf.RBF_OK
        check_answer(h)
        assert 0 < int(h.accepted.sum()) < 20  # some are taken and some are not


def test_gradient_of_a_distillation_through_a_quantised_head():
    with rbf.Ops(64, 2048, stream=torch.cuda.current_stream()) as o:
        h = Head(o, 7, 4, 1500, 256, seed=2)
        h.learn()
        assert o.check_device_error() == rbf.RBF_OK
        scores = h.target.view(-1, h.vocab)
        want, want_grad = ref.distill(scores=scores.cpu(), index=h.index.cpu(), teacher=h.teacher.cpu(), rest=None, weight=None, temperature=2.0)
        loss_error, rel = ref.distill_errors(scores.cpu(), h.teacher.cpu(), 2.0, None)
        assert bool(((h.loss.cpu().double() - want).abs() <= loss_error + want.abs() * 2.0 ** -22).all())
        q = torch.softmax(scores.cpu().double() / 2.0, 1)
        allowed = 2.0 * 4 * rel * (q + (want_grad / 2.0).abs()) + want_grad.abs() * 2.0 ** -8
        assert bool(((h.grad.cpu().double() - want_grad).abs() <= allowed).all())
        dx, size = ref.product(h.grad8, h.grad_scale, h.wt8, h.wt_scale, 128)
        assert bool(((h.dx.double() - dx).abs() <= ref.product_error(size, h.vocab, torch.float32, dx)).all())
        # and against the unquantised product: a quantised number is off by half a step of its mantissa, or of its block's smallest number
        g8 = h.grad.double().abs() * 2.0 ** -3 + ref.spread(h.grad_scale, 1, *h.grad.shape) * 2.0 ** -17
        w8 = h.wt.double().abs() * 2.0 ** -4 + ref.spread(h.wt_scale, 128, *h.wt.shape) * 2.0 ** -10
        allowed = g8 @ h.wt.double().abs().t() + h.grad.double().abs() @ w8.t() + g8 @ w8.t()
        assert bool(((h.dx.double() - h.grad.double() @ h.wt.double().t()).abs() <= allowed * 1.001).all())


def test_captured_and_replayed():
    """Two graphs of one handle, replayed in turn: they share its workspace, one after the other on its stream."""
    s = torch.cuda.Stream()
    with rbf.Ops(64, 2048, stream=s) as o:
        h = Head(o, 6, 3, 1100, 384, seed=3)
        with torch.cuda.stream(s):
            h.clear()
            h.answer()
            h.learn()
            want = h.outputs()
            graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
            for graph, step in zip(graphs, (h.answer, h.learn)):
                with torch.cuda.graph(graph, stream=s):
                    step()
            for order in ((0, 1), (1, 0, 0, 1, 0)):
                h.clear()
                for i in order:
                    graphs[i].replay()
                got = h.outputs()
                torch.cuda.synchronize()
                assert same(got, want)
            # what was written into the inputs since then is read
            h.x.copy_(h.x.flip(0))
            graphs[0].replay()
            replayed = h.outputs()
            h.answer()
            assert same(h.outputs(), replayed) and not torch.equal(replayed[2], want[2])
        torch.cuda.synchronize()
        assert o.check_device_error() == rbf.RBF_OK


def test_two_handles_at_once():
    streams = [torch.cuda.Stream() for _ in range(2)]
    handles = [rbf.Ops(64, 2048, stream=s) for s in streams]
    try:
        heads = [Head(o, 6, 3, 1200, 256, seed=4 + i) for i, o in enumerate(handles)]
        wants = []
        for h, s in zip(heads, streams):
            with torch.cuda.stream(s):
                h.clear()
                h.answer()
                h.learn()
                wants.append(h.outputs())
            torch.cuda.synchronize()
        for _ in range(3):
            for h, s in zip(heads, streams):
                with torch.cuda.stream(s):
                    h.clear()
            for _ in range(4):
                for h, s in zip(heads, streams):
                    with torch.cuda.stream(s):
                        h.answer()
                        h.learn()
            torch.cuda.synchronize()
            assert all(same(h.outputs(), w) for h, w in zip(heads, wants))
        assert all(o.check_device_error() == rbf.RBF_OK for o in handles)
    finally:
        for o in handles:
            o.close()


def test_sizes_drawn_at_random():
    g = torch.Generator()
    g.manual_seed(9)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    with rbf.Ops(256, 2048, stream=torch.cuda.current_stream()) as o:
        for i in range(6):
            check = Head(o, pick(1, 9), pick(1, 6), pick(200, 900), pick(1, 700), seed=20 + i)
            check.answer()
            check_answer(check)
        assert o.check_device_error() == rbf.RBF_OK


def test_launches_and_failed_launches():
    with rbf.Ops(64, 2048, stream=torch.cuda.current_stream()) as o:
        h = Head(o, 3, 2, 500, 256, seed=5)
        h.answer()
        calls = {
            "quantise": (lambda: o.quantize_f8_dev(h.x, h.x8, h.x_scale), 1),
            "product": (lambda: o.matmul_f8_dev(h.x8, h.x_scale, h.w8, h.w_scale, h.target.view(-1, h.vocab)), 1),
            "verify": (lambda: o.verify_dev(h.target, h.drafted, h.u, h.token, h.accepted, d_draft=h.draft), 2),
            "distil": (lambda: o.distill_dev(h.target.view(-1, h.vocab), h.index, h.teacher, d_loss=h.loss), 1),
        }
        for name, (call, launches) in calls.items():
            call()
            assert o.last_launches == launches, name
            before = h.outputs()
            o.inject_host_fault(launches)
            with pytest.raises(rbf.RbfError):
                call()
            o.inject_host_fault(0)
            call()
            assert same(h.outputs(), before), name
        assert o.check_device_error() == rbf.RBF_OK


def test_product_of_unaligned_rows_of_more_than_the_workspace_holds():
    """Rows of b off 16-byte boundaries are put on them 32 MB at a time."""
    g = gen(6)
    m, n, k = 5, 5000, 8001
    a8, b8 = torch.empty(m, k, dtype=E4M3, device="cuda"), torch.empty(n, k, dtype=E4M3, device="cuda")
    a_scale, b_scale = torch.empty(m, 63, device="cuda"), torch.empty(40, 63, device="cuda")
    with rbf.Ops(8, 8192, stream=torch.cuda.current_stream()) as o:
        o.quantize_f8_dev(torch.randn(m, k, generator=g, device="cuda"), a8, a_scale)
        o.quantize_f8_dev(torch.randn(n, k, generator=g, device="cuda"), b8, b_scale, block_rows=128)
        out = torch.empty(m, n, device="cuda")
        o.matmul_f8_dev(a8, a_scale, b8, b_scale, out)
        assert o.last_launches == 5  # a's rows, and two parts of b's
        want, size = ref.product(a8, a_scale, b8, b_scale, 128)
        assert bool(((out.double() - want).abs() <= ref.product_error(size, k, torch.float32, want)).all())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantise_a_row_that_ends_at_2_to_the_31(block_rows):
    cols = 2 ** 31 - 1
    x = torch.zeros(1, cols, dtype=torch.bfloat16, device="cuda")
    g = gen(7)
    tail, head = torch.randn(1, 255, generator=g, device="cuda").bfloat16(), torch.randn(1, 256, generator=g, device="cuda").bfloat16()
    x[:, -255:], x[:, :256] = tail, head
    q, scale = torch.full((1, cols), 9, dtype=torch.uint8, device="cuda"), torch.full((1, 2 ** 24), -1.0, device="cuda")
    with rbf.Ops(1, 64, stream=torch.cuda.current_stream()) as o:
        o.quantize_f8_dev(x, q.view(E4M3), scale, block_rows=block_rows)
    for part, at, blocks in ((tail, slice(cols - 255, cols), slice(2 ** 24 - 2, 2 ** 24)), (head, slice(0, 256), slice(0, 2))):
        want, want_scale = ref.quantize_f8(part, E4M3, block_rows)
        assert torch.equal(q[:, at].view(E4M3).double(), want) and torch.equal(scale[:, blocks], want_scale)
    assert bool((scale[:, 2:-2] == 0).all())
    for i in range(256, cols - 255, 2 ** 28):
        assert not bool(q[:, i:min(i + 2 ** 28, cols - 255)].any())


def test_rows_whose_offsets_pass_32_bits():
    """The last rows of views that span more than 2^32 bytes."""
    ld, rows, k = 2 ** 26, 70, 300
    g = gen(8)
    with rbf.Ops(128, 512, stream=torch.cuda.current_stream()) as o:
        near = torch.randn(rows, k, generator=g, device="cuda").bfloat16()
        far = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)[:, :k]
        far.copy_(near)
        space8 = torch.empty(rows * ld, dtype=torch.uint8, device="cuda").view(rows, ld)
        far8, near8 = space8[:, :k].view(E4M3), torch.empty(rows, k, dtype=E4M3, device="cuda")
        far_scale, near_scale = torch.empty(rows, 3, device="cuda"), torch.empty(rows, 3, device="cuda")
        o.quantize_f8_dev(far, far8, far_scale)
        o.quantize_f8_dev(near, near8, near_scale)
        assert torch.equal(far8.view(torch.uint8), near8.view(torch.uint8)) and torch.equal(far_scale, near_scale)
        want = torch.empty(rows, rows, dtype=torch.bfloat16, device="cuda")
        o.matmul_f8_dev(near8, near_scale, near8, near_scale, want)
        o.matmul_f8_dev(far8, near_scale, far8, near_scale, far[:, :rows])
        assert torch.equal(far[:, :rows], want)
        # the same rows as scores
        far.copy_(near * 3)
        scores = torch.empty(rows, k + 4, dtype=torch.bfloat16, device="cuda")[:, :k]  # on 16-byte boundaries, as those are: sums in the same order
        scores.copy_(far)
        index, teacher = torch.arange(rows, device="cuda", dtype=torch.int32)[:, None] % k, torch.ones(rows, 1, device="cuda")
        losses, grad = torch.empty(2, rows, device="cuda"), torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
        o.distill_dev(scores, index, teacher, d_loss=losses[0], d_grad=grad)
        drafted = torch.randint(0, k, (7, 9), generator=g, device="cuda", dtype=torch.int32)
        u = torch.rand(7, 10, generator=g, device="cuda")
        got = []
        for t in (scores.unflatten(0, (7, 10)), far.unflatten(0, (7, 10)), (near * 3).view(7, 10, k)):
            token, accepted, logprob = torch.empty(7, 10, dtype=torch.int32, device="cuda"), torch.empty(7, dtype=torch.int32, device="cuda"), torch.empty(7, 10, device="cuda")
            o.verify_dev(t, drafted, u, token, accepted, d_logprob=logprob, d_draft=t[:, :9])
            got.append((token, accepted, logprob))
        assert same(*got[:2])
        # rows that lie otherwise on 16-byte boundaries are summed in another order: the logarithms' last bits
        assert same(got[0][:2], got[2][:2]) and bool(((got[0][2] == got[2][2]) | ((got[0][2] - got[2][2]).abs() <= 2.0 ** -18)).all())
        o.distill_dev(far, index, teacher, d_loss=losses[1], d_grad=far)  # in place
        assert torch.equal(losses[0], losses[1]) and torch.equal(far, grad)
        assert o.check_device_error() == rbf.RBF_OK


@pytest.mark.parametrize("dtype,rows,vocab", [(torch.float32, 3, 1001), (torch.bfloat16, 400, 515), (torch.float16, 2, 70001), (torch.bfloat16, 1, 1_100_003)])
def test_gradient_in_the_scores_place(dtype, rows, vocab):
    g = gen(rows)
    scores = torch.randn(rows, vocab, generator=g, device="cuda").to(dtype)
    index = torch.randint(0, vocab, (rows, 5), generator=g, device="cuda", dtype=torch.int32)
    teacher = torch.randn(rows, 5, generator=g, device="cuda")
    losses, grad = torch.empty(2, rows, device="cuda"), torch.empty_like(scores)
    with rbf.Ops(1, 64, stream=torch.cuda.current_stream()) as o:
        o.distill_dev(scores, index, teacher, d_loss=losses[0], d_grad=grad)
        o.distill_dev(scores, index, teacher, d_loss=losses[1], d_grad=scores)
    assert torch.equal(losses[0], losses[1]) and torch.equal(scores, grad)


def test_weight_multiplies_loss_and_gradient():
    g = gen(10)
    scores = torch.randn(4, 300, generator=g, device="cuda")
    index, teacher = torch.arange(12, device="cuda", dtype=torch.int32).view(4, 3) * 7, torch.randn(4, 3, generator=g, device="cuda")
    weight = torch.tensor([1.0, -2.0, math.nan, 0.5], device="cuda")
    losses, grads = torch.empty(2, 4, device="cuda"), torch.empty(2, 4, 300, device="cuda")
    with rbf.Ops(1, 64, stream=torch.cuda.current_stream()) as o:
        o.distill_dev(scores, index, teacher, d_loss=losses[0], d_grad=grads[0])
        o.distill_dev(scores, index, teacher, d_loss=losses[1], d_grad=grads[1], weight=weight)
    for i, w in enumerate(weight.tolist()):
        if math.isnan(w):
            assert bool(losses[1, i].isnan()) and bool(grads[1, i].isnan().all())
        else:
            assert float(losses[1, i]) == float(losses[0, i]) * w
            # the factor is rounded with the weight in it, or without: powers of two change no bit
            assert torch.equal(grads[1, i], grads[0, i] * w)
