"""Plain implementations of the scoring-head operators on the CPU, in whole
numbers and 64-bit floats, for the tests."""
import math

import numpy as np

LOG2E = np.float32(1.4426950408889634)
ONE = 1 << 36    # the largest weight of a row
PARTS = 1 << 30  # steps of u and of top_p

# Relative error of a weight computed in fp32: z = (x - top) * rate has two
# roundings of 2^-24 each and the rate one more, |z| <= 37 where the weight is
# not zero, and 2^z turns an error of z into one of ln 2 times it; exp2f adds
# 2 units of 2^-23. Weights and their sum each carry it.
WEIGHT_ERROR = 2 * (37 * 3 * 2.0 ** -24 * math.log(2) + 2 * 2.0 ** -23)


def quantize(x):
    """(q, scale) of quantize_rows_i8_dev: float32 arithmetic, one rounding a step."""
    x = np.asarray(x, np.float32)
    q = np.zeros(x.shape, np.int8)
    scale = np.zeros(x.shape[0], np.float32)
    for i, row in enumerate(x):
        t = np.max(np.abs(row)) if row.size else np.float32(0)
        if not np.isfinite(t):
            scale[i] = np.nan
            continue
        scale[i] = t * (np.float32(1) / np.float32(127))
        if t > 0:
            pre = np.float32(2.0 ** 100 if t < 2.0 ** -100 else 1.0)
            q[i] = np.rint((row * pre) * ((np.float32(1) / (t * pre)) * np.float32(127))).astype(np.int8)
    return q, scale


def product_sums(a, b):
    """Exact sums of the 8-bit product: float64 holds them (below 2^53)."""
    return (a.astype(np.float64) @ b.astype(np.float64).T).astype(np.int64)


def _order(x):
    """Indices in the search's order: higher score first, lower index on a tie (a NaN is -infinity, -0 is 0)."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64)) + 0.0
    return np.lexsort((np.arange(x.size), -x)), x


def sample_exact(x, u, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of a row of whole-numbered scores at temperature log2(e) in float32, where every weight is a
    power of two: whole numbers throughout."""
    order, x = _order(np.asarray(x))
    if x.size == 0 or x[order[0]] == -np.inf:
        return -1, -math.inf
    top = x[order[0]]
    w = np.array([ONE >> int(min(top - v, 63)) if v > -np.inf and v != top else (ONE if v == top else 0) for v in x], dtype=object)
    # 2^-37 is half of the smallest weight and rounds to even: to zero.
    keep = list(order[:top_k] if 0 < top_k < x.size else order)
    if top_p < 1:
        target = sum(w[j] for j in keep) * int(np.rint(np.float32(max(top_p, 0.0)) * np.float32(PARTS))) // PARTS
        upto, short = 0, []
        for j in keep:
            if short and upto >= target:
                break
            short.append(j)
            upto += w[j]
        keep = short
    keep = [j for i, j in enumerate(keep) if i == 0 or float(w[j]) / ONE >= np.float32(min_p)]
    keep.sort()
    total = sum(w[j] for j in keep)
    aim = total * min(int(np.floor(np.float32(max(u, 0.0)) * np.float32(PARTS))), PARTS - 1) // PARTS
    upto = 0
    for j in keep:
        upto += w[j]
        if upto > aim:
            return int(j), math.log(w[j] / total)
    raise AssertionError("no index")


def sample_allowed(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """{token: its possible logprobs} that 64-bit arithmetic allows within the error of fp32 weights: more than one only
    where u, or a threshold, is that near to a boundary."""
    order, x = _order(np.asarray(x))
    if x.size == 0 or x[order[0]] == -np.inf:
        return {-1: [-math.inf]}
    top = x[order[0]]
    warm = temperature > 0
    k = 1 if not warm else (top_k if 0 < top_k < x.size else x.size)
    keep = order[:k]
    z = x[keep] - top
    w = np.where(z == 0, 1.0, np.exp(z / (temperature if warm else 1.0)))
    w[w < 2.0 ** -37] = 0.0
    eps = WEIGHT_ERROR
    upto = np.cumsum(w)

    def count(p):  # the fewest that reach p of the sum
        return 1 + int((upto[:-1] < p * upto[-1]).sum())

    counts = {k}
    if top_p < 1:
        p = max(float(np.float32(top_p)), 0.0)
        counts = set(range(count(p - eps), count(p + eps) + 1))
    mins = [0.0]
    if min_p > 0:
        near = w[(np.abs(w - float(np.float32(min_p))) <= eps * w)]
        mins = [float(np.float32(min_p))] + [m * f for m in near for f in (1 - eps, 1 + eps)]
    allowed = {}
    for n in counts:
        for m in mins:
            kept = np.array([j for i, j in enumerate(keep[:n]) if i == 0 or w[i] >= m])
            kept.sort()
            wk = np.where(x[kept] == top, 1.0, np.exp((x[kept] - top) / (temperature if warm else 1.0)))
            edge = np.concatenate([[0.0], np.cumsum(wk)]) / wk.sum()
            uc = min(max(float(np.float32(u)), 0.0), 1 - 2.0 ** -30)
            for i in np.nonzero((edge[:-1] - eps <= uc) & (uc < edge[1:] + eps) & (wk >= 2.0 ** -37))[0]:
                allowed.setdefault(int(kept[i]), []).append(math.log(wk[i] / wk.sum()))
    return allowed
