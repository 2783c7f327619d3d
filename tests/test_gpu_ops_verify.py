"""Verification of drafted tokens (include/rbf_ops.h, verify_dev) against the definition in 64 bits."""
import math

import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import more_ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(4096, 64, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == rbf.RBF_OK


def case(seqs, drafts, vocab, dtype=torch.float32, seed=0, near=0.7, with_draft=True):
    g = torch.Generator()
    g.manual_seed(seed * 1000 + seqs * 31 + drafts * 7 + vocab)
    target = torch.randn(seqs, drafts + 1, vocab, generator=g) * 2.5
    draft = target[:, :drafts] + near * torch.randn(seqs, drafts, vocab, generator=g)
    target, draft = target.to(dtype), draft.to(dtype)
    noise = -torch.log(-torch.log(torch.rand(seqs, drafts, vocab, generator=g).clamp(1e-20, 1 - 1e-7)))
    tokens = (draft.float() + noise).argmax(-1).int() if vocab else torch.zeros(seqs, drafts, dtype=torch.int32)
    u = torch.rand(seqs, drafts + 1, generator=g)
    return {"target": target, "draft": draft if with_draft else None, "tokens": tokens, "u": u, "count": None, "temperature": None}


def call(ops, c, target=None, draft=None):
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    seqs, places, _ = c["target"].shape
    token = torch.full((seqs, places), 77, dtype=torch.int32, device="cuda")
    accepted = torch.full((seqs,), 77, dtype=torch.int32, device="cuda")
    logprob = torch.full((seqs, places), 77.0, device="cuda")
    ops.verify_dev(cu(c["target"]) if target is None else target, cu(c["tokens"]), cu(c["u"]), token, accepted, d_logprob=logprob,
                   d_draft=cu(c["draft"]) if draft is None else draft, draft_count=cu(c["count"]), temperature=cu(c["temperature"]))
    return token.cpu(), accepted.cpu(), logprob.cpu()


def check(ops, c):
    got = call(ops, c)
    ref.check_verify(c["target"], c["draft"], c["tokens"], c["count"], c["u"], c["temperature"], *got)
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("seqs,drafts,vocab", [(1, 0, 5), (1, 1, 1), (1, 4, 1000), (3, 1, 2), (7, 3, 17), (5, 7, 4099), (40, 5, 1001), (2, 2, 100003),
                                               (1, 15, 33), (2, 40, 130)])
def test_sizes(ops, dtype, seqs, drafts, vocab):
    check(ops, case(seqs, drafts, vocab, dtype))


@pytest.mark.parametrize("vocab", [1, 9, 1000, 50001])
def test_without_draft_scores(ops, vocab):
    c = case(20, 3, vocab, torch.bfloat16, seed=2, with_draft=False)
    c["tokens"][::2] = c["target"][::2, :3].float().argmax(-1).int()  # some that are likely
    check(ops, c)


def test_every_number_of_accepted_tokens(ops):
    c = case(64, 6, 300, seed=3, near=0.5)
    _, accepted, _ = check(ops, c)
    assert set(accepted.tolist()) == set(range(7))


def test_counts_temperatures_and_masks(ops):
    c = case(48, 5, 777, torch.float16, seed=4)
    g = torch.Generator()
    g.manual_seed(9)
    c["count"] = torch.randint(-1, 8, (48,), generator=g, dtype=torch.int32)  # clamped to 0 .. 5
    c["temperature"] = torch.tensor([0.0, 1.0, 0.3, 2.5, -1.0, math.nan, 1e-30, math.inf] * 6)
    c["target"][torch.rand(48, 6, 777, generator=g) < 0.5] = -math.inf
    c["draft"][torch.rand(48, 5, 777, generator=g) < 0.1] = -math.inf
    c["target"][3, 0] = -math.inf
    c["target"][8, 2:] = -math.inf
    c["target"][16, :, 5:] = -math.inf
    c["target"][24, 1, :] = torch.finfo(torch.float16).min
    c["target"][25, 0, 7] = math.nan
    c["target"][26, 0, :] = math.nan
    c["target"][27, 0, 9] = math.inf
    c["target"][28, 1, 3:6] = math.inf
    c["draft"][29, 0, 4] = math.inf
    c["draft"][30, 0, :] = -math.inf
    check(ops, c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("base,heat", [(3e4, 0.7), (-3e4, 0.7), (45000.0, 1.0), (46000.0, 1.0), (-46000.0, 1.0), (1e6, 1.0), (3.0, 1e-5), (-1e30, 1e25),
                                       (0.0, 1e-20), (0.0, 1e20), (0.0, 1e-36)])
def test_scores_far_from_zero(ops, dtype, base, heat):
    """Largest scores over T on either side of 2^16, where weights are taken without a difference of scores and with one."""
    c = case(9, 3, 1003, seed=int(abs(base)) % 97)
    c["target"], c["draft"] = ((base + heat * c[k].double()).to(dtype) for k in ("target", "draft"))
    c["temperature"] = torch.full((9,), heat)
    check(ops, c)


def test_what_is_not_needed_is_not_looked_at(ops):
    """Places behind a sequence's drafted tokens hold anything, and so do the draft's scores of a greedy one."""
    c = case(6, 4, 500, seed=5)
    c["count"] = torch.tensor([0, 1, 2, 3, 4, 2], dtype=torch.int32)
    c["temperature"] = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 0.0])
    first = check(ops, c)
    for b, n in enumerate(c["count"].tolist()):
        c["target"][b, n + 1:] = math.nan
        c["draft"][b, n:] = math.inf
        c["tokens"][b, n:] = -5
    c["draft"][5] = math.nan
    for x, y in zip(first, call(ops, c)):
        assert torch.equal(x, y)


def test_tokens_outside_of_the_vocabulary(ops):
    for with_draft in (True, False):
        c = case(4, 2, 100, seed=6, with_draft=with_draft)
        c["tokens"][0, 0], c["tokens"][1, 0], c["tokens"][2, 0] = -1, 100, 2 ** 31 - 1
        _, accepted, _ = check(ops, c)
        assert accepted[:3].tolist() == [0, 0, 0]


def test_equal_rows_accept_everything(ops):
    c = case(30, 4, 1003, torch.bfloat16, seed=7, near=0.0)
    c["u"][:, :4] = 1 - 2.0 ** -24  # nearer to 1 than two fp32 sums of the same weights in another order have to be (2^-23 each): either way
    check(ops, c)
    c["u"][:, :4] = 1 - 2.0 ** -16
    _, accepted, _ = check(ops, c)
    assert bool((accepted == 4).all())


def test_random_numbers_at_their_ends(ops):
    c = case(30, 3, 301, seed=8)
    c["u"][:10] = 0.0
    c["u"][10:20] = 1 - 2.0 ** -24
    c["u"][20:, -1] = 1.0  # clamped
    check(ops, c)


def test_disjoint_rows(ops):
    """The draft has no mass where the target has: the first token is refused, the answer drawn from all of p."""
    c = case(16, 1, 64, seed=9)
    c["target"][:, 0, ::2] = -math.inf
    c["draft"][:, 0, 1::2] = -math.inf
    c["tokens"][:, 0] = 2 * (c["tokens"][:, 0] // 2)
    token, accepted, _ = check(ops, c)
    assert bool((accepted == 0).all()) and bool((token[:, 0] % 2 == 1).all())


def test_strides_and_offsets(ops):
    """Padded places and sequences, rows that start anywhere, and a draft that lies otherwise than the target."""
    for dtype in (torch.float32, torch.bfloat16):
        c = case(5, 3, 1021, dtype, seed=10)
        want = call(ops, c)
        wide = torch.full((5, 6, 1040), math.inf, dtype=dtype, device="cuda")
        target = wide[:, 1:5, 3:1024]
        target.copy_(c["target"])
        other = torch.full((5, 3, 1029), math.inf, dtype=dtype, device="cuda")[:, :, 6:1027]
        other.copy_(c["draft"])
        got = call(ops, c, target, other)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # the same fp32 weights summed in the order of other 16-byte vectors: either sum is within RATIO_ERROR of the exact one
        assert torch.equal(got[2].isinf(), want[2].isinf())
        assert bool(((got[2] - want[2]).abs().nan_to_num(0.0) <= 2 * ref.RATIO_ERROR + want[2].abs().nan_to_num(0.0, 0.0, 0.0) * 2.0 ** -22).all())


def test_distribution_is_the_targets():
    """Over many random numbers the first answered token has the target's distribution, whatever the draft's: a
    share of n draws is off by less than 5 standard deviations (one in 10^6 of them is not)."""
    n, vocab = 20000, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    row = torch.tensor([2.0, 1.0, 0.0, -1.0, 1.5, -math.inf, 0.5, -3.0], device="cuda")
    q_row = torch.tensor([0.0, 2.0, 0.5, 0.0, -1.0, 1.0, 0.0, 1.0], device="cuda")
    p, q = torch.softmax(row.double(), 0), torch.softmax(q_row.double(), 0)
    tokens = torch.multinomial(q.float(), n, replacement=True, generator=g).int()[:, None]
    token, accepted = torch.empty(n, 2, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    with rbf.Ops(2 * n, 1, stream=torch.cuda.current_stream()) as ops:
        ops.verify_dev(row.expand(n, 2, vocab).contiguous(), tokens, torch.rand(n, 2, generator=g, device="cuda"), token, accepted,
                       d_draft=q_row.expand(n, 1, vocab).contiguous())
        share = torch.bincount(token[:, 0].long(), minlength=vocab).double() / n
    assert bool(((share - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all()), share
    assert abs(float(accepted.double().mean()) - float(torch.minimum(p, q).sum())) < 5 * 0.5 / n ** 0.5


def test_long_row(ops):
    """A vocabulary whose rows do not fit the cluster's shared memory, with ties over all of it."""
    vocab = 1_700_001
    c = case(1, 1, 8, seed=11)
    g = torch.Generator()
    g.manual_seed(3)
    c["target"] = torch.randint(-3, 4, (1, 2, vocab), generator=g).float()
    c["draft"] = torch.randint(-3, 4, (1, 1, vocab), generator=g).float()
    c["tokens"] = torch.tensor([[int(c["target"][0, 0].argmin())]], dtype=torch.int32)
    for k in range(4):
        c["u"] = torch.rand(1, 2, generator=g)
        check(ops, c)


def test_same_bits_again_and_in_a_graph(ops):
    c = case(9, 5, 3001, torch.bfloat16, seed=12)
    first = call(ops, c)
    for x, y in zip(first, call(ops, c)):
        assert torch.equal(x, y)
    target, draft, tokens, u = (c[k].cuda() for k in ("target", "draft", "tokens", "u"))
    token, accepted = torch.empty(9, 6, dtype=torch.int32, device="cuda"), torch.empty(9, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    with rbf.Ops(64, 64, stream=s) as o:
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            o.verify_dev(target, tokens, u, token, accepted, d_draft=draft)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                o.verify_dev(target, tokens, u, token, accepted, d_draft=draft)
            for _ in range(3):
                token.fill_(0)
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(token.cpu(), first[0]) and torch.equal(accepted.cpu(), first[1])
        u.uniform_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        c["u"] = u.cpu()
        want = call(ops, c)
        assert torch.equal(token.cpu(), want[0]) and torch.equal(accepted.cpu(), want[1])


def test_empty_calls(ops):
    c = case(0, 3, 10)
    ops.verify_dev(c["target"].cuda(), c["tokens"].cuda(), c["u"].cuda(), torch.empty(0, 4, dtype=torch.int32, device="cuda"),
                   torch.empty(0, dtype=torch.int32, device="cuda"))
    assert ops.last_launches == 0
    c = case(2, 1, 0)
    token, accepted, logprob = call(ops, c)
    assert bool((token == -1).all()) and bool((accepted == 0).all()) and bool((logprob == -math.inf).all())
