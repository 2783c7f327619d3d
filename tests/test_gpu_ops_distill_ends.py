"""Distillation (include/rbf_ops.h, distill_dev) at the ends of its range: long rows of like scores, listed scores at the
type's lowest value, NaN beside nothing but masked scores."""
import math

import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests.test_gpu_ops_distill import call, case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(64, 64, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == rbf.RBF_OK


@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 2 ** 26), (torch.float32, 9_000_001), (torch.bfloat16, 2 ** 26 - 5), (torch.float16, 1_100_003)])
@pytest.mark.parametrize("gap", [0.0625, 0.15625, 0.34375, 0.8125, 1.28125])
def test_sums_of_long_rows(ops, dtype, vocab, gap):
    """A quarter of the scores at 0 and three quarters at -gap, so that every thread adds the same number over and over and
    its roundings do not cancel; one listed score that has about a quarter of the mass. In 2^-20 of itself the mass of the others
    is off by 0.25 and 0.13 (the exponential; its argument's two roundings, |z| < 2), 0.57 (six additions of four vectors, three
    of those in a piece), 0.75 (twelve joins of threads' sums by half a step of 2^-23), 0.25 and 0.69 (the factor below the listed
    score: the exponential; half a step of its argument, |z| < 32) and 0.2 (log2(e) in fp32): less than 2.9 in all, of which the
    loss takes three quarters. A gradient has 0.38 of its own weight, 1.7 of the others' sum, a quarter of 2.9 and five
    roundings, 0.31: less than 3.2."""
    a = torch.full((vocab,), -gap, dtype=dtype, device="cuda")
    a[::4] = 0.0
    n0 = -(-vocab // 4)
    at = 4 * (n0 // 2)
    others = (n0 - 1) + (vocab - n0) * math.exp(-gap)
    a[at] = math.log(others / 3)
    listed = float(a[at].double())
    whole = others + math.exp(listed)
    index, teacher = torch.tensor([[at]], dtype=torch.int32, device="cuda"), torch.zeros(1, 1, device="cuda")
    loss, grad = torch.empty(1, device="cuda"), torch.empty(1, vocab, dtype=dtype, device="cuda")
    ops.distill_dev(a[None], index, teacher, d_loss=loss, d_grad=grad)
    want = math.log(whole) - listed
    assert abs(float(loss[0]) - want) <= 0.75 * 2.9 * 2.0 ** -20 + want * 2.0 ** -23, (float(loss[0]), want)
    half = torch.finfo(dtype).eps / 2 + 3.2 * 2.0 ** -20
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    for j, e in ((0, 1.0), (1, math.exp(-gap)), (vocab - 1, 1.0 if (vocab - 1) % 4 == 0 else math.exp(-gap))):
        assert abs(float(grad[0, j]) - e / whole) <= e / whole * half + tiny, j
    want = math.exp(listed) / whole - 1
    assert abs(float(grad[0, at]) - want) <= abs(want) * half


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("temperature,weight", [(0.5, 1.0), (0.7, 1.0), (2.0, 1 / 512), (1.0, 1e-3), (2.0 ** -20, 1.0), (2.0 ** 20, 2.0 ** -30), (0.3, 1e-30)])
def test_listed_scores_at_the_lowest_value(ops, dtype, temperature, weight):
    """A listed score at the type's lowest value makes a large loss, T weight p of it, which is a number wherever that is one:
    whatever T, on the way there."""
    c = case(6, 700, 3, dtype, seed=30, temperature=temperature)
    lowest = torch.finfo(dtype).min
    c["weight"] = torch.full((6,), weight)
    c["teacher"] = (torch.tensor([[4.0, 0.0, -1.0]]) * min(temperature, 1.0)).to(dtype).repeat(6, 1)  # p of about 0.98, 0.02 and less
    c["scores"].scatter_(1, c["index"][:, :1].long(), lowest)
    c["scores"][2].fill_(1.0)
    c["scores"][2].scatter_(0, c["index"][2].long(), lowest)             # all of the list
    c["scores"][3, int(c["index"][3, 0])] = 1.0
    c["scores"][3, int(c["index"][3, 2])] = lowest                       # an unlikely one alone
    c["scores"][4].clamp_(-2, 2)
    c["scores"][4, int(c["index"][4, 1])] = torch.finfo(dtype).max       # and another as far away as can be
    c["scores"][4, int(c["index"][4, 0])] = lowest
    c["rest"] = torch.full((6,), -2.0)
    want = torch.zeros(6, dtype=torch.float64)
    for i in range(6):  # by logarithms throughout: a mass 1e38 below the largest score has one, but is no 64-bit number
        z, at = c["scores"][i].double() / temperature, c["index"][i].long()
        outside = torch.ones(700, dtype=torch.bool).scatter(0, at, False)
        logq = torch.cat([z[at], torch.logsumexp(z[outside], 0)[None]]) - torch.logsumexp(z, 0)
        logp = torch.log_softmax(torch.cat([c["teacher"][i].double() / temperature, c["rest"][i:i + 1].double()]), 0)
        want[i] = float(c["weight"][i]) * temperature ** 2 * (logp.exp() * (logp - logq)).sum()
    loss, grad = (t.cpu().double() for t in call(ops, c))
    assert bool(torch.isfinite(grad).all())
    fits = want.abs() < 3.4e38
    assert bool(fits[:4].all())
    # the products p (t - s) / T and their sum in pairs of fp32 numbers, p to 2^-19, and the last factors' roundings
    assert bool(((loss - want).abs() <= want.abs() * 2.0 ** -18)[fits].all()), (loss, want)
    assert bool((loss == math.inf)[~fits].all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_not_a_number_beside_masked_scores(ops, dtype):
    """Where every score outside of the list is -infinity, a NaN in the list, the teacher's logits, its rest or the weight
    makes the whole row's gradient NaN all the same."""
    c = case(7, 300, 4, dtype, seed=31, weighted=True)
    for i in range(7):
        row = c["scores"][i].clone()
        c["scores"][i] = -math.inf
        c["scores"][i, c["index"][i].long()] = row[c["index"][i].long()]
    c["rest"] = torch.full((7,), -math.inf)
    c["scores"][0, int(c["index"][0, 1])] = math.nan
    c["scores"][1, int(c["index"][1, 1])] = math.inf
    c["teacher"][2, 3] = math.nan
    c["teacher"][3, 0] = math.inf
    c["rest"][4] = math.nan
    c["weight"][5] = math.nan
    loss, grad = call(ops, c)
    assert bool(loss[:6].isnan().all()) and bool(grad[:6].isnan().all())
    assert bool(torch.isfinite(loss[6])) and bool(torch.isfinite(grad[6]).all())
    outside = torch.ones(300, dtype=torch.bool)
    outside[c["index"][6].long()] = False
    assert bool((grad[6].cpu()[outside] == 0).all())
