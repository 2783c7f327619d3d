"""Distillation (include/rbf_ops.h, distill_dev) against the definition in 64 bits and against differences."""
import math

import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests import more_ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(64, 64, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == rbf.RBF_OK


def case(rows, vocab, k, dtype=torch.float32, seed=0, rest=False, weighted=False, temperature=1.0):
    g = torch.Generator()
    g.manual_seed(seed * 977 + rows * 31 + vocab * 3 + k)
    full = torch.randn(rows, vocab, generator=g) * 2.5
    scores = (full + torch.randn(rows, vocab, generator=g)).to(dtype)
    teacher, index = full.topk(k, dim=1) if k else (torch.zeros(rows, 0), torch.zeros(rows, 0, dtype=torch.int64))
    order = torch.rand(rows, k, generator=g).argsort(1)  # in any order
    teacher, index = teacher.gather(1, order).to(dtype), index.gather(1, order).int()
    r = torch.logsumexp((full / temperature).scatter(1, index.long(), -math.inf), 1) if rest else None
    w = torch.rand(rows, generator=g) if weighted else None
    return {"scores": scores, "index": index, "teacher": teacher, "rest": r, "weight": w, "temperature": temperature}


def call(ops, c, with_loss=True, with_grad=True, scores=None, grad=None):
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    loss = torch.full((len(c["scores"]),), 77.0, device="cuda") if with_loss else None
    if grad is None and with_grad:
        grad = torch.full(c["scores"].shape, 77.0, dtype=c["scores"].dtype, device="cuda")
    ops.distill_dev(cu(c["scores"]) if scores is None else scores, cu(c["index"]), cu(c["teacher"]), d_loss=loss, d_grad=grad, rest=cu(c["rest"]),
                    weight=cu(c["weight"]), temperature=c["temperature"])
    return loss, grad


def check(ops, c):
    loss, grad = (t.cpu().double() for t in call(ops, c))
    want, want_grad = ref.distill(**c)
    dtype = c["scores"].dtype
    loss_error, rel = ref.distill_errors(c["scores"], c["teacher"], c["temperature"], c["weight"])
    same = (loss == want) | (loss.isnan() & want.isnan())
    assert bool((same | ((loss - want).abs() <= loss_error + want.abs() * 2.0 ** -22)).all()), (loss, want, loss_error)
    w = (torch.ones(len(loss)) if c["weight"] is None else c["weight"].abs()).double()[:, None] * c["temperature"]
    # q and each p are off by `rel`; what stands between them is at most 1, and is rounded to the type
    q = torch.softmax(torch.where(c["scores"].isnan(), -math.inf, c["scores"].double()) / c["temperature"], 1).nan_to_num(0.0)
    terms = q + (want_grad / w.clamp_min(1e-30)).abs()
    allowed = w * 4 * rel * terms + want_grad.abs() * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert torch.equal(grad.isnan(), want_grad.isnan())
    off = (grad - want_grad).abs().nan_to_num(0.0)
    assert bool((off <= allowed).all() if not want_grad.isnan().any() else (off <= allowed.nan_to_num(math.inf)).all()), float((off / allowed).max())
    return loss, grad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (1, 2, 1), (3, 17, 5), (5, 1000, 8), (2, 4099, 64), (40, 257, 257), (300, 65, 3), (1, 100003, 50),
                                          (2, 70001, 1024), (600, 40, 0)])
@pytest.mark.parametrize("rest", [False, True])
def test_sizes(ops, dtype, rows, vocab, k, rest):
    check(ops, case(rows, vocab, k, dtype, rest=rest, weighted=True))


@pytest.mark.parametrize("temperature", [0.5, 2.0, 7.3, 100.0])
def test_temperatures(ops, temperature):
    check(ops, case(6, 900, 20, rest=True, temperature=temperature))
    check(ops, case(6, 900, 20, torch.bfloat16, temperature=temperature))


def test_gradient_is_the_losses_difference(ops):
    """Central differences of the 64-bit loss of nearby scores, which are off by their third derivative, h^2 / 6 of at most 1."""
    c = case(3, 12, 4, rest=True, weighted=True, temperature=1.7)
    _, grad = check(ops, c)
    h = 1e-4
    for i in range(3):
        for j in range(12):
            up, down = (dict(c, scores=c["scores"].double().clone()) for _ in range(2))
            up["scores"][i, j] += h
            down["scores"][i, j] -= h
            slope = float(ref.distill(**up)[0][i] - ref.distill(**down)[0][i]) / (2 * h)
            assert abs(slope - float(grad[i, j])) <= 1e-6, (i, j)


def test_entries_that_are_missing_or_come_twice(ops):
    c = case(8, 300, 12, seed=2, rest=True)
    c["index"][0, 3:] = -1
    c["index"][1, :] = -1
    c["index"][2, 5] = 300
    c["index"][3, 0] = 2 ** 31 - 1
    c["index"][4, 1] = c["index"][4, 0]
    c["index"][5, :] = 7
    c["index"][6, 2:9] = c["index"][6, 9]
    c["teacher"][7, 4] = -math.inf
    check(ops, c)
    c["rest"] = None
    loss, grad = check(ops, c)
    assert float(loss[1]) == 0 and bool((grad[1] == 0).all())  # no teacher
    for dtype in (torch.bfloat16, torch.float16):
        check(ops, dict(c, scores=c["scores"].to(dtype)))


def test_same_index_over_and_over_gives_the_same_bits(ops):
    c = case(4, 50, 40, seed=3)
    c["index"] = c["index"] % 5
    first = call(ops, c)
    for _ in range(5):
        again = call(ops, c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    check(ops, c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_and_weights(ops, dtype):
    c = case(12, 500, 10, dtype, seed=4, rest=True, weighted=True)
    g = torch.Generator()
    g.manual_seed(1)
    c["scores"][torch.rand(12, 500, generator=g) < 0.3] = -math.inf
    c["scores"].scatter_(1, c["index"].long(), c["teacher"])
    c["scores"][0] = -math.inf                          # nothing is left
    c["weight"][1] = 0.0                                # a padded row, with anything in it
    c["scores"][1] = math.nan
    keep = torch.zeros(500, dtype=torch.bool)
    keep[c["index"][2].long()] = True
    c["scores"][2][~keep] = -math.inf                   # nothing outside of the list, but a teacher's rest there
    c["scores"][3][keep.new_zeros(500).scatter(0, c["index"][3].long(), True)] = -math.inf  # nothing in the list
    c["scores"][4] = torch.finfo(dtype).min             # all of the type's lowest value
    c["scores"][5][int(c["index"][5, 0])] = -math.inf   # one of the list
    c["rest"][6] = -math.inf
    loss, grad = check(ops, c)
    assert float(loss[0]) == 0 and bool((grad[0] == 0).all()) and float(loss[1]) == 0 and bool((grad[1] == 0).all())
    assert float(loss[2]) == math.inf and float(loss[3]) == math.inf and float(loss[5]) == math.inf


def test_not_a_number_makes_a_row_so(ops):
    c = case(8, 200, 6, seed=5, rest=True)
    inside, outside = c["index"][:, 0].long(), [next(j for j in range(200) if j not in r.tolist()) for r in c["index"]]
    c["scores"][0, outside[0]] = math.nan
    c["scores"][1, inside[1]] = math.nan
    c["scores"][2, outside[2]] = math.inf
    c["scores"][3, inside[3]] = math.inf
    c["teacher"][4, 2] = math.nan
    c["teacher"][5, 1] = math.inf
    c["rest"][6] = math.nan
    loss, grad = call(ops, c)
    assert bool(loss[:7].isnan().all()) and bool(grad[:7].isnan().all())
    assert bool(torch.isfinite(loss[7])) and bool(torch.isfinite(grad[7]).all())


def test_far_apart_masses(ops):
    """Listed and other scores that are hundreds apart: what is small keeps its bits."""
    for gap in (-300.0, -40.0, 40.0, 300.0):
        c = case(3, 64, 4, seed=6, rest=True)
        c["scores"].scatter_add_(1, c["index"].long(), torch.full((3, 4), gap))
        check(ops, c)
        c["rest"] = c["rest"] + gap
        check(ops, c)


def test_loss_and_gradient_apart(ops):
    c = case(9, 3000, 16, torch.bfloat16, seed=7, rest=True, weighted=True)
    loss, grad = call(ops, c)
    assert torch.equal(call(ops, c, with_grad=False)[0], loss)
    assert torch.equal(call(ops, c, with_loss=False)[1], grad)
    call(ops, c, with_loss=False, with_grad=False)
    assert ops.last_launches == 0


def test_strides_and_offsets(ops):
    for dtype in (torch.float32, torch.bfloat16):
        for shift, other in ((0, 0), (3, 3), (1, 2), (5, 0)):
            c = case(5, 1003, 9, dtype, seed=8, rest=True)
            loss, grad = call(ops, c)
            wide = torch.full((5, 1040), math.inf, dtype=dtype, device="cuda")[:, shift:shift + 1003]
            wide.copy_(c["scores"])
            whole = torch.full((5, 1040), 5.0, dtype=dtype, device="cuda")
            out = whole[:, other:other + 1003]
            got, _ = call(ops, c, scores=wide, grad=out)
            # the same numbers in other vectors: sums in another order
            assert bool(((got - loss).abs() <= 2.0 ** -18).all())
            assert bool(((out.double() - grad.double()).abs() <= 2.0 ** -18 + grad.double().abs() * torch.finfo(dtype).eps).all())
            assert bool((whole[:, :other] == 5.0).all()) and bool((whole[:, other + 1003:] == 5.0).all())


def test_types_of_the_teacher(ops):
    for kind in (torch.float32, torch.bfloat16, torch.float16):
        c = case(4, 300, 7, torch.bfloat16, seed=9)
        c["teacher"] = c["teacher"].to(kind)
        check(ops, c)
        c["scores"] = c["scores"].float()
        check(ops, c)


@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 300_001), (torch.bfloat16, 1_100_003)])
def test_rows_in_pieces(ops, dtype, vocab):
    """Rows that sixteen CTAs do not hold at a time."""
    c = case(1, vocab, 33, dtype, seed=10, rest=True)
    c["index"][0, 5] = c["index"][0, 6]
    check(ops, c)


def test_in_a_graph(ops):
    c = case(7, 2000, 11, torch.bfloat16, seed=11, weighted=True)
    want = call(ops, c)
    dev = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
    loss, grad = torch.empty(7, device="cuda"), torch.empty_like(dev["scores"])
    s = torch.cuda.Stream()
    with rbf.Ops(64, 64, stream=s) as o:
        torch.cuda.synchronize()
        go = lambda: o.distill_dev(dev["scores"], dev["index"], dev["teacher"], d_loss=loss, d_grad=grad, weight=dev["weight"])  # noqa: E731
        with torch.cuda.stream(s):
            go()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                go()
            grad.zero_()
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])


def test_teacher_is_a_search(ops):
    """The lists that a search returns, as they are: int32 indices and fp32 scores, -1 where there is no entry."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    corpus, queries = torch.randn(5000, 64, generator=g, device="cuda"), torch.randn(6, 64, generator=g, device="cuda")
    student = torch.randn(6, 5000, generator=g, device="cuda")
    with rbf.Engine(5000, 64, 16, max_batch=6, flags=rbf.RBF_FLAG_BF16_CORPUS) as e:
        e.upload_corpus_rowmajor(corpus)
        idx, sc = e.search_resident_batch(queries.cpu().numpy(), 16)
    c = {"scores": student.cpu(), "index": torch.from_numpy(idx.copy()).int(), "teacher": torch.from_numpy(sc.copy()), "rest": None, "weight": None, "temperature": 4.0}
    check(ops, c)
