"""The plain implementations that the GPU tests of the scoring-head operators
compare with, checked against cases worked out by hand."""
import math

import numpy as np

from tests import ops_reference as ref


def test_quantize_by_hand():
    x = np.array([[0, 0, 0], [127, -63.5, 0.5], [1, np.inf, 0], [2.0 ** -140, -2.0 ** -141, 0]], np.float32)
    q, s = ref.quantize(x)
    assert q.tolist() == [[0, 0, 0], [127, -64, 0], [0, 0, 0], [127, -64, 0]]  # 63.5 and 0.5 go to even
    assert s[0] == 0 and s[1] == 1 and np.isnan(s[2]) and s[3] > 0


def test_sample_exact_by_hand():
    x = np.array([1.0, 3.0, 3.0, -np.inf, 2.0])          # weights 1/4 1 1 0 1/2
    assert ref.sample_exact(x, 0.0)[0] == 0
    assert ref.sample_exact(x, 0.25 / 2.75 + 1e-4)[0] == 1
    assert ref.sample_exact(x, 0.999)[0] == 4
    assert ref.sample_exact(x, 0.999, top_k=1) == (1, 0.0)    # the lower index of the tie
    assert ref.sample_exact(x, 0.999, top_k=2)[0] == 2
    assert ref.sample_exact(x, 0.999, top_p=0.5)[0] == 2      # 1 of 2.75 does not reach half
    assert ref.sample_exact(x, 0.999, min_p=0.6)[0] == 2
    assert ref.sample_exact(x, 0.999, min_p=2.0) == (1, 0.0)  # the best index always stays
    assert ref.sample_exact(np.full(3, -np.inf), 0.5) == (-1, -math.inf)


def test_the_two_sampling_references_agree():
    rng = np.random.default_rng(3)
    for _ in range(200):
        x = rng.integers(-20, 5, rng.integers(1, 60)).astype(np.float64)
        ask = dict(top_k=int(rng.integers(0, 20)), top_p=float(rng.choice([1.0, rng.random()])),
                   min_p=float(rng.choice([0.0, 0.1 * rng.random()])))
        u = float(np.float32(rng.random()))
        token, logprob = ref.sample_exact(x, u, **ask)
        allowed = ref.sample_allowed(x, u, temperature=1 / math.log(2), **ask)
        assert token in allowed and min(abs(lp - logprob) for lp in allowed[token]) < 1e-9
