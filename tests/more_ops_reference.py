"""What 8-bit floating-point rows and their product, verification of drafted tokens and distillation compute, in 64
bits (include/rbf_ops.h), written apart from the kernels, and how far those may be off by their arithmetic."""
import math

import torch

F8 = {torch.float8_e4m3fn: (448.0, 3, -6), torch.float8_e5m2: (57344.0, 2, -14)}  # largest, mantissa bits, lowest exponent


# ------------------------------------------------------------------ 8 bits


def round_f8(y, dtype):
    """Values (64 bits, within the type's range) to the nearest numbers of an 8-bit type, halves to even."""
    top, bits, low = F8[dtype]
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -60))).clamp_min(low)
    e = torch.where(torch.exp2(e) > y.abs(), (e - 1).clamp_min(low), e)  # a logarithm rounded up
    step = torch.exp2(e - bits)
    return (torch.round(y / step) * step).clamp(-top, top)


def quantize_f8(x, dtype, block_rows):
    """The 8-bit numbers as 64-bit ones, with the arithmetic of the definition: each step in fp32."""
    top = F8[dtype][0]
    rows, cols = x.shape
    x = x.float()
    r_blocks, c_blocks = -(-rows // block_rows), -(-cols // 128)
    q, scale = torch.zeros(rows, cols, dtype=torch.float64, device=x.device), torch.zeros(r_blocks, c_blocks, device=x.device)
    for i in range(r_blocks):
        for j in range(c_blocks):
            at = (slice(i * block_rows, min(rows, (i + 1) * block_rows)), slice(128 * j, min(cols, 128 * j + 128)))
            b = x[at]
            t = b.abs().max()
            if not bool(torch.isfinite(b).all()):
                scale[i, j] = math.nan
            elif float(t) > 0:
                most, one = torch.tensor(top, device=x.device), torch.tensor(1.0, device=x.device)
                inv = (one / t) * most
                scale[i, j] = t * (one / most)
                if float(inv) > 2.0 ** 127:
                    inv, scale[i, j] = torch.tensor(2.0 ** 127, device=x.device), 2.0 ** -127
                q[at] = round_f8((b * inv).double(), dtype)
    return q, scale


def spread(scale, block_rows, rows, cols):
    r, c = torch.arange(rows, device=scale.device) // block_rows, torch.arange(cols, device=scale.device) // 128
    return scale.double()[r][:, c]


def product(a, a_scale, b, b_scale, block_rows, bias=None):
    """The product in 64 bits, and the sum of its terms' magnitudes."""
    x = a.double() * spread(a_scale, 1, *a.shape)
    y = b.double() * spread(b_scale, block_rows, *b.shape)
    out, size = x @ y.t(), x.abs() @ y.abs().t()
    return (out, size) if bias is None else (out + bias.double(), size + bias.double().abs())


def product_error(size, depth, dtype, out):
    """How far a product may be off: 32 products of an instruction are aligned and summed, an accumulator of 24 bits
    takes four such sums a block; a step each for the scales' product, for its product with the sum, for the blocks' sum
    and the bias, of at most a whole step of fp32 (2^-23), and half a step of the output's type."""
    steps = 32 + 4 + 3 + -(-depth // 128) + 1
    return size * (steps * 2.0 ** -23) + out.abs() * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).tiny


# ----------------------------------------------------------- verification


def shares(x, temperature):
    """softmax(x / T) in 64 bits by the definition's rules for NaN, infinities and T; zeros where nothing is left."""
    x = torch.where(torch.isnan(x), -math.inf, x.double())
    top = x.max() if x.numel() else torch.tensor(-math.inf, dtype=torch.float64)
    if top == -math.inf:
        return torch.zeros_like(x)
    if not temperature > 0:
        p = torch.zeros_like(x)
        p[int(torch.nonzero(x == top)[0])] = 1.0
        return p
    if top == math.inf:
        w = (x == math.inf).double()
    elif temperature == math.inf:
        w = (x > -math.inf).double()
    else:
        w = torch.exp((x - top) / temperature)
    return w / w.sum()


# Of a probability ratio: sums of weights that are off by 2^-22 (the exponential) and by 2^-24 for each of |z| (its
# argument) with |z| below 60 where it matters.
RATIO_ERROR = 2.0 ** -20
# Of a draw's running sum, in shares of p's whole: each probability is held to 2^-29, and p - q has two of them.
DRAW_ERROR = 2.0 ** -28


def check_verify(target, draft, tokens, count, u, temperature, token, accepted, logprob):
    """The answers of one call, place by place, on the CPU: every decision has to be the definition's, up to the errors above."""
    seqs, places, vocab = target.shape
    for b in range(seqs):
        heat = 1.0 if temperature is None else float(temperature[b])
        n = places - 1 if count is None else min(max(int(count[b]), 0), places - 1)
        got = int(accepted[b])
        assert 0 <= got <= n, (b, got)
        for i in range(got + 1):
            p = shares(target[b, i], heat)
            if i < n:
                x = int(tokens[b, i])
                inside = 0 <= x < vocab
                if draft is None or not heat > 0:
                    q = torch.zeros_like(p)
                    if inside:
                        q[x] = 1.0
                else:
                    q = shares(draft[b, i], heat)
                px, qx = (float(p[x]), float(q[x])) if inside else (0.0, 1.0)
                lhs = float(u[b, i]) * qx if heat > 0 else (0.0 if px > 0 else 1.0)
                if i < got:
                    assert inside and px > 0 and lhs < px * (1 + RATIO_ERROR), (b, i, lhs, px)
                    assert int(token[b, i]) == x
                else:
                    assert not inside or px == 0 or lhs >= px * (1 - RATIO_ERROR), (b, i, lhs, px)
                if i < got:
                    check_logprob(logprob, b, i, px)
                    continue
            x = int(token[b, i])
            if float(p.sum()) == 0:
                assert x == -1 and (logprob is None or float(logprob[b, i]) == -math.inf)
                continue
            left = p
            if i < n and heat > 0:
                left = (p - q).clamp_min(0) if inside or draft is not None else p
                if float(left.sum()) < DRAW_ERROR:
                    left = p
            assert 0 <= x < vocab, (b, i, x)
            upto = left.cumsum(0)
            r = min(math.floor(max(float(u[b, -1]), 0.0) * 2 ** 30), 2 ** 30 - 1) * 2.0 ** -30 * float(upto[-1]) if heat > 0 else 0.0
            assert float(upto[x]) > r - DRAW_ERROR and float(upto[x] - left[x]) <= r + DRAW_ERROR, (b, i, x, r)
            assert float(p[x]) > 0
            check_logprob(logprob, b, i, float(p[x]))
        for i in range(got + 1, places):
            assert int(token[b, i]) == -1 and (logprob is None or float(logprob[b, i]) == -math.inf)


def check_logprob(logprob, b, i, px):
    """A logarithm of a sum (RATIO_ERROR) less a score's distance, rounded to fp32."""
    if logprob is not None:
        want = math.log(px)
        assert abs(float(logprob[b, i]) - want) <= 2 * RATIO_ERROR + abs(want) * 2.0 ** -21, (b, i, float(logprob[b, i]), want)


# ----------------------------------------------------------- distillation


def distill(scores, index, teacher, rest=None, weight=None, temperature=1.0):
    """Loss and gradient in 64 bits, a row at a time."""
    rows, vocab = scores.shape
    loss = torch.zeros(rows, dtype=torch.float64)
    grad = torch.zeros(rows, vocab, dtype=torch.float64)
    for i in range(rows):
        w = 1.0 if weight is None else float(weight[i])
        here = [e for e in range(index.shape[1]) if 0 <= int(index[i, e]) < vocab]
        at = [int(index[i, e]) for e in here]
        z = scores[i].double() / temperature
        tau = torch.cat([teacher[i][here].double() / temperature, torch.full((1,), -math.inf, dtype=torch.float64) if rest is None else rest[i:i + 1].double()])
        if w == 0 or bool((tau == -math.inf).all()) or bool((z == -math.inf).all()):
            continue
        p, q = torch.softmax(tau, 0), torch.softmax(z, 0)
        outside = torch.ones(vocab, dtype=torch.bool)
        outside[at] = False
        logq_all, logp = torch.log_softmax(z, 0), torch.log_softmax(tau, 0)  # below the largest: a logarithm vanishes beside 1e38
        q_rest = torch.exp(logq_all[outside]).sum()
        logq = torch.cat([logq_all[at], torch.log(q_rest)[None]])
        loss[i] = w * temperature ** 2 * torch.where(p > 0, p * (logp - logq), torch.where(torch.isnan(p), p, 0.0)).sum()
        g = q.clone()
        if bool((z[outside] > -math.inf).any()):
            g[outside] = torch.softmax(z[outside], 0) * (q_rest - p[-1])
        for e, j in enumerate(at):
            g[j] = g[j] - p[e]
        grad[i] = w * temperature * g
    return loss, grad


def distill_errors(scores, teacher, temperature, weight=None):
    """How far a row's loss and each of its gradients' terms may be off. A weight 2^z is off by 2^-22 (the exponential)
    and by z's two roundings, 2^-23 |z| ln 2, |z| <= 60 where it counts for anything; a sum of them by as much and its
    roundings, 2^-21 in all. So a logarithm of a sum has an error of `rel`; a loss has two, and the products p (t - s) / T
    with roundings of 2^-22 of their size."""
    rel = 2.0 ** -22 + 60 * 2.0 ** -23 * math.log(2) + 2.0 ** -21
    finite = torch.where(torch.isfinite(scores.double()), scores.double(), 0.0)
    far = (finite.abs().amax(1) + torch.where(torch.isfinite(teacher.double()), teacher.double(), 0.0).abs().amax(1) if teacher.shape[1] else finite.abs().amax(1)) / temperature
    w = torch.ones(len(scores), dtype=torch.float64) if weight is None else weight.double().abs()
    return w * temperature ** 2 * (4 * rel + far * 2.0 ** -22), rel
