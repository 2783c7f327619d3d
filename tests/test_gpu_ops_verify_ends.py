"""Verification of drafted tokens (include/rbf_ops.h, verify_dev) at the ends of its range: rows with +infinity, random
numbers of 0, scores further apart than the largest fp32 number, rows that agree but for rounding."""
import math

import pytest
import torch

import resident_brute_force_gb300 as rbf
from tests.test_gpu_ops_verify import case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    with rbf.Ops(4096, 64, stream=torch.cuda.current_stream()) as o:
        yield o
        assert o.check_device_error() == rbf.RBF_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [50, 20011])
@pytest.mark.parametrize("u", [0.25, 0.999])
def test_tokens_beside_an_infinite_score_have_no_mass(ops, dtype, vocab, u):
    """Where a target's row holds +infinity a token with a finite score is refused, whatever the draft says of it."""
    c = case(8, 2, vocab, dtype, seed=20)
    c["u"][:, :2] = u
    c["tokens"][:, 0] = 3
    c["target"][:7, 0, 7] = math.inf
    c["draft"][0, 0, 3] = -math.inf                  # the draft has no mass on the token
    c["draft"][1, 0, 3] = math.nan
    c["draft"][2, 0, 9] = math.inf                   # nor here, beside its own +infinity
    c["draft"][3, 0, 3] = math.inf                   # all of it
    c["draft"][4, 0] = -math.inf                     # its row is empty
    c["tokens"][5, 0] = 7                            # the one score that counts: accepted
    c["tokens"][6, 0], c["draft"][6, 0, 7] = 7, -math.inf
    c["target"][7, 0], c["draft"][7, 0, 3] = -math.inf, -math.inf  # an empty row accepts nothing
    token, accepted, _ = check(ops, c)
    assert accepted[[0, 1, 2, 3, 4, 7]].tolist() == [0] * 6 and int(accepted[5]) > 0 and int(accepted[6]) > 0
    assert token[:5, 0].tolist() == [7] * 5 and int(token[7, 0]) == -1
    _, accepted, _ = check(ops, dict(c, draft=None))
    assert accepted[[0, 1, 2, 3, 4, 7]].tolist() == [0] * 6


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_random_number_of_zero_accepts_any_probability(ops, dtype):
    """0 < p(x) however far p(x) lies below q(x); where p(x) is 0 the token is refused."""
    c = case(9, 2, 300, dtype, seed=21)
    c["tokens"][:, 0] = 11
    c["u"][:, 0] = 0.0
    c["u"][8, 0] = -0.0
    c["temperature"] = torch.full((9,), 0.02)
    c["target"][:, 0].clamp_(-9.0, 2.0)
    c["draft"][:, 0].clamp_(-9.0, 2.0)
    c["draft"][:, 0, 11] = 2.0
    for i, gap in enumerate((1.0, 3.0, 3.6, 5.0, 9.0, 12.0)):  # over T: 50 to 600, 2^-72 to 2^-866
        c["target"][i, 0, 5], c["target"][i, 0, 11] = 2.0, 2.0 - gap
    c["target"][6, 0, 11] = -math.inf
    c["target"][7, 0, 5] = math.inf
    _, accepted, _ = check(ops, c)
    assert bool((accepted[:6] > 0).all()) and accepted[6:8].tolist() == [0, 0] and int(accepted[8]) > 0
    c["u"][:, 0] = 2.0 ** -126  # above 0: refused from about there on
    _, accepted, _ = check(ops, c)
    assert int(accepted[0]) > 0 and accepted[1:8].tolist() == [0] * 7


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heat", [2e36, 1e37, 1e38, 3e38, math.inf])
@pytest.mark.parametrize("vocab", [9, 40, 3001])
def test_scores_further_apart_than_the_largest_number(ops, dtype, heat, vocab):
    """x - max passes fp32's range, x / T - max / T does not: those scores have their weight."""
    c = case(12, 3, vocab, dtype, seed=22)
    for k in ("target", "draft"):
        c[k] = (c[k].double() / 2.5 * 1.5e38).clamp(-3.38e38, 3.38e38).to(dtype)  # a good part of them at either end
    c["target"][0, 0, 2:] = -math.inf
    c["target"][0, 0, 0], c["target"][0, 0, 1] = torch.finfo(dtype).max, torch.finfo(dtype).min
    c["target"][1, 0, ::3] = torch.finfo(dtype).min
    c["draft"][2, 0, 1::3] = torch.finfo(dtype).max
    c["target"][3, 1, 4] = math.inf
    c["temperature"] = torch.full((12,), heat)
    check(ops, c)
    check(ops, dict(c, draft=None))
    for u in (0.0, 0.3, 0.9, 1 - 2.0 ** -24):
        c["u"][:, -1] = u
        check(ops, c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0.0, 0.5, 3.0, -20.0, 96.0])
def test_rows_that_agree_but_for_rounding(ops, dtype, shift):
    """A draft's row that is the target's plus a constant has the same probabilities: behind a token outside of the
    vocabulary the answer is drawn from p, not from what rounding leaves of p - q."""
    c = case(40, 1, 4001, torch.float32, seed=23)
    c["target"] = ((c["target"] * 8).round() / 8).to(dtype)  # eighths: the sum below is exact in fp32
    c["draft"] = (c["target"][:, :1].double() + shift).to(dtype)
    if dtype == torch.bfloat16 and shift:
        same = c["draft"].double() == c["target"][:, :1].double() + shift
        c["draft"][~same], c["target"][:, :1][~same] = -math.inf, -math.inf
    c["tokens"][:, 0] = -1
    c["temperature"] = torch.linspace(0.3, 2.0, 40)
    _, accepted, _ = check(ops, c)
    assert bool((accepted == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heat", [0.02, 1.0, 3.0])
def test_masks_of_the_lowest_value(ops, dtype, heat):
    """A score at the type's lowest value has a probability of 0, as in 64 bits: its token is refused whatever the random
    number and the draft's own mask; a row that holds nothing else has equal ones."""
    c = case(8, 2, 500, dtype, seed=24)
    lowest = torch.finfo(dtype).min
    c["temperature"] = torch.full((8,), heat)
    c["tokens"][:, 0] = 13
    c["u"][:, 0] = 0.5
    c["u"][0, 0] = 0.0
    c["target"][:4, 0, 13] = lowest                       # 0: u = 0
    c["draft"][1, 0, 13] = lowest                         # masked on both sides
    c["draft"][2, 0, 13], c["target"][2, 0, 13] = lowest / 2, lowest  # less so on the draft's
    c["draft"][3, 0, 13] = -math.inf
    c["draft"][4, 0, 13] = lowest                         # on the draft's alone: accepted
    c["target"][5, 0], c["draft"][5, 0] = lowest, lowest  # all of either row: equal probabilities
    c["u"][6, 0], c["target"][6, 0, 13], c["target"][6, 0, 0] = 0.0, -700 * heat, 0.0  # 2^-1010, but for the row's own largest
    c["target"][6, 0, 1:13], c["target"][6, 0, 14:] = -1.0, -1.0
    token, accepted, _ = check(ops, c)
    assert accepted[:4].tolist() == [0] * 4 and bool((accepted[4:7] > 0).all())
    assert bool((token[:4, 0] != 13).all())
    _, accepted, _ = check(ops, dict(c, draft=None))
    assert accepted[:4].tolist() == [0] * 4
