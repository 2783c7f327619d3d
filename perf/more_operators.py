"""More scoring-head operators as measured cases: rows and blocks quantised to 8-bit floating point, their product with
a scale for each block of 128, drafted tokens verified against the target's scores, and distillation from a teacher's
best logits with its gradient.

`run` computes a case in its plain form (elementary torch operations) or, where `own` is true, with the calls a
user makes of this package. The sizes are those of this repository's corpora, batches and layers (10k to 1M rows of
384 to 1024 values, batches of 1 to 256, layers of 4,096 and more for ingest) with odd and ragged ones among them.

What the operators compute (MAX = 448 for e4m3, 57344 for e5m2):

  quantise   of each block (128 values of a row, or of 128 rows): t = max |x|, scale = t / MAX, q = the nearest 8-bit
             number to x * (MAX / t)
  product    out[i, j] = sum over blocks c of a_scale[i, c] * b_scale[j or j / 128, c] * sum_{k in c} a[i, k] b[j, k] (+ bias[j])
  verify     p = softmax(target / T), q = softmax(draft / T) (no draft scores: all of it on the drafted token); token x of
             position i is accepted if u_i q_i(x) < p_i(x); at the first one that is not, the answer is drawn from
             max(0, p_i - q_i), after the last one from p (first index at which the running sum passes u times the sum)
  distill    p = softmax of the teacher's k logits / T and, where it has one, the logarithm of its remaining mass;
             q = softmax(scores / T); loss = T^2 (sum p_e log(p_e / q_e) + p_rest log(p_rest / q_rest)), and its gradient;
             loss and gradient are multiplied by the row's weight
"""
import math

import torch

own = False

_FLOAT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
_handle = None


def _ops():
    """The handle (workspace and stream) that a user's program creates once and keeps."""
    global _handle
    if _handle is None:
        import resident_brute_force_gb300 as rbf
        _handle = rbf.Ops(16384, 8192, stream=torch.cuda.current_stream())
    return _handle


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one query embedding, quantised before it is scored
        {"name": "quantise 1x768", "op": "quantise", "rows": 1, "cols": 768, "dtype": "f32", "f8": "e4m3", "block": 1},
        # a wide layer's weights, a scale for each block of 128 x 128
        {"name": "quantise 8192x8192", "op": "quantise", "rows": 8192, "cols": 8192, "dtype": "bf16", "f8": "e4m3", "block": 128},
        # decoding: one token through a wide layer
        {"name": "product 1x32000x4096", "op": "product", "m": 1, "n": 32000, "k": 4096, "dtype": "bf16", "block": 128, "a8": "e4m3", "bias": False},
        # a ragged batch on a ragged vocabulary, every channel with scales of its own
        {"name": "product 37x10007x1000", "op": "product", "m": 37, "n": 10007, "k": 1000, "dtype": "f16", "block": 1, "a8": "e4m3", "bias": True},
        # the full batch of queries against the 1M-row corpus
        {"name": "product 256x1000000x768", "op": "product", "m": 256, "n": 1000000, "k": 768, "dtype": "bf16", "block": 1, "a8": "e4m3", "bias": False},
        # many tokens at once (ingest, or a prompt)
        {"name": "product 4096x8192x4096", "op": "product", "m": 4096, "n": 8192, "k": 4096, "dtype": "bf16", "block": 128, "a8": "e4m3", "bias": False},
        # one sequence, a few drafted tokens on a small vocabulary: latency
        {"name": "verify 1x4x10000", "op": "verify", "seqs": 1, "drafts": 4, "vocab": 10000, "dtype": "f32", "mode": "plain"},
        # a ragged batch: other lengths and temperatures a sequence, masked scores, a greedy and a fully masked one among them
        {"name": "verify 61x5x100003", "op": "verify", "seqs": 61, "drafts": 5, "vocab": 100003, "dtype": "bf16", "mode": "mixed"},
        # the full batch on a large vocabulary
        {"name": "verify 64x7x128000", "op": "verify", "seqs": 64, "drafts": 7, "vocab": 128000, "dtype": "bf16", "mode": "plain"},
        # one row's loss (evaluation) on the small corpus' lists of 8
        {"name": "distill 1x10000", "op": "distill", "rows": 1, "vocab": 10000, "k": 8, "dtype": "f32", "mode": "loss", "temperature": 1.0},
        # a ragged training batch with the teacher's remaining mass, short lists, masked scores and rows without weight
        {"name": "distill 509x100003", "op": "distill", "rows": 509, "vocab": 100003, "k": 50, "dtype": "f16", "mode": "mixed", "temperature": 2.0},
        # a training batch on a large vocabulary: loss and gradient
        {"name": "distill 4096x128000", "op": "distill", "rows": 4096, "vocab": 128000, "k": 64, "dtype": "bf16", "mode": "grad", "temperature": 1.0},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "product", "verify", "verify", "distill", "distill"])
    if op == "quantise":
        rows, cols = _spread(rng, 1, 8192), _spread(rng, 16, 8192)
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["f32", "bf16", "f16"]) if rows * cols < 1 << 25 else "bf16",
                "f8": rng.choice(["e4m3", "e4m3", "e5m2"]), "block": rng.choice([1, 128])}
    if op == "product":
        m, k = _spread(rng, 1, 4096), _spread(rng, 64, 8192)
        n = _spread(rng, 64, max(64, min(1000000, 768000000 // k, 256000000 // m, (1 << 37) // (m * k))))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["f32", "bf16", "f16"]) if m * n < 1 << 26 else "bf16", "block": rng.choice([1, 128]),
                "a8": rng.choice(["e4m3", "e4m3", "e5m2"]), "bias": rng.random() < 0.5}
    if op == "verify":
        drafts = rng.randint(1, 15)
        seqs = _spread(rng, 1, min(128, 512 // (drafts + 1)))
        vocab = _spread(rng, 64, min(300000, 65536000 // (seqs * (drafts + 1))))
        return {"op": op, "seqs": seqs, "drafts": drafts, "vocab": vocab, "dtype": rng.choice(["f32", "bf16", "f16"]) if seqs * drafts * vocab < 1 << 25 else "bf16",
                "mode": rng.choice(["plain", "plain", "mixed", "mixed", "none"])}
    rows = _spread(rng, 1, 4096)
    vocab = _spread(rng, 64, min(300000, 524288000 // rows))
    return {"op": op, "rows": rows, "vocab": vocab, "k": min(vocab, _spread(rng, 1, 256)), "dtype": rng.choice(["f32", "bf16", "f16"]) if rows * vocab < 1 << 27 else "bf16",
            "mode": rng.choice(["loss", "grad", "grad", "mixed"]), "temperature": rng.choice([1.0, 1.0, 2.0, 0.7])}


# ----------------------------------------------------------------- inputs


def _pitched(rows, cols, dtype):
    """[rows, cols] in rows whose start is a multiple of 16 bytes, as the resident corpora are laid out."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def _embeddings(g, rows, cols, dtype):
    """Values with a few dominant directions and rows of different size, as embeddings and activations have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    x *= torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
    out = _pitched(rows, cols, dtype)
    out.copy_(x)
    return out


def _f8_rows(g, rows, cols, kind):
    """8-bit rows of which each block's largest number is near the type's, as quantised rows have them."""
    dtype, top = _F8[kind]
    q = _pitched(rows, cols, dtype)
    for r in range(0, rows, 1 << 17):  # a block at a time: the values before rounding are not all held at once
        n = min(1 << 17, rows - r)
        q[r:r + n].copy_((torch.randn(n, cols, generator=g, device="cuda") * (top / 3.0)).clamp_(-top, top))
    return q


def _scales(g, *shape):
    return torch.exp(0.5 * torch.randn(*shape, generator=g, device="cuda")) * 0.001


def _scores(g, dtype, *shape):
    """Scores of a vocabulary: a broad bulk and a few likely ones."""
    x = 2.5 * torch.randn(*shape, generator=g, device="cuda")
    few = torch.randint(0, shape[-1], (*shape[:-1], min(40, shape[-1])), generator=g, device="cuda")
    x.scatter_add_(-1, few, 6.0 * torch.rand(few.shape, generator=g, device="cuda"))
    return x if dtype is None else x.to(dtype)


def _blocks(n):
    return -(-n // 128)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if own:
        s["ops"] = _ops()
    op = case["op"]
    if op == "quantise":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _embeddings(g, rows, cols, _FLOAT[case["dtype"]])
        s["q"] = _pitched(rows, cols, _F8[case["f8"]][0])
        s["scale"] = torch.empty(-(-rows // case["block"]), _blocks(cols), device="cuda")
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_scale"] = _f8_rows(g, m, k, case["a8"]), _scales(g, m, _blocks(k))
        s["b"], s["b_scale"] = _f8_rows(g, n, k, "e4m3"), _scales(g, -(-n // case["block"]), _blocks(k))
        s["bias"] = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        s["out"] = torch.empty(m, n, dtype=_FLOAT[case["dtype"]], device="cuda")
    elif op == "verify":
        seqs, drafts, vocab, mode = case["seqs"], case["drafts"], case["vocab"], case["mode"]
        dtype, mixed = _FLOAT[case["dtype"]], mode == "mixed"
        target = _scores(g, None, seqs, drafts + 1, vocab)
        draft = target[:, :drafts] + 0.5 * torch.randn(seqs, drafts, vocab, generator=g, device="cuda")  # a smaller model of the same text
        u = lambda lo, hi, *n: lo + (hi - lo) * torch.rand(*n, generator=g, device="cuda")  # noqa: E731
        s["temperature"] = u(0.6, 1.2, seqs)
        s["count"] = None
        if mixed:
            kinds = torch.randint(0, 6, (seqs,), generator=g, device="cuda")
            s["temperature"] = torch.where(kinds == 0, 0.0, s["temperature"])  # greedy
            s["count"] = torch.randint(0, drafts + 1, (seqs,), generator=g, device="cuda", dtype=torch.int32)
            mask = torch.rand(seqs, 1, vocab, generator=g, device="cuda") < 0.25  # an output grammar's
            target.masked_fill_(mask, -math.inf)
            if seqs > 2:
                target[seqs // 2] = -math.inf
        warm = torch.where(s["temperature"] > 0, s["temperature"], 1.0)[:, None, None]
        noise = -torch.log(-torch.log(torch.rand(seqs, drafts, vocab, generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)))
        s["tokens"] = (draft / warm + noise).argmax(-1).int()  # drawn from the draft
        s["target"], s["draft"] = target.to(dtype), None if mode == "none" else draft.to(dtype)
        s["u"] = torch.rand(seqs, drafts + 1, generator=g, device="cuda")
        s["token"], s["logprob"] = torch.empty(seqs, drafts + 1, dtype=torch.int32, device="cuda"), torch.empty(seqs, drafts + 1, device="cuda")
        s["accepted"] = torch.empty(seqs, dtype=torch.int32, device="cuda")
    else:
        rows, vocab, k, dtype = case["rows"], case["vocab"], case["k"], _FLOAT[case["dtype"]]
        s["scores"] = torch.empty(rows, vocab, dtype=dtype, device="cuda")
        s["index"], s["teacher"] = torch.empty(rows, k, dtype=torch.int32, device="cuda"), torch.empty(rows, k, dtype=dtype, device="cuda")
        rest = torch.empty(rows, device="cuda")
        for r in range(0, rows, 512):  # the teacher's whole rows are not kept
            n = min(512, rows - r)
            t = _scores(g, None, n, vocab)
            s["scores"][r:r + n].copy_(t.add(torch.randn(n, vocab, generator=g, device="cuda")).sub_(1.0))
            best, at = t.topk(k, dim=1)
            s["teacher"][r:r + n].copy_(best)
            s["index"][r:r + n].copy_(at)
            rest[r:r + n] = torch.logsumexp(t.div_(case["temperature"]).scatter_(1, at, -math.inf), 1)
        # the mean over the batch; gradients of type f16 with a loss scale, as their range asks for
        mean = (2.0 ** 14 if dtype == torch.float16 else 1.0) / rows
        s["rest"], s["weight"] = None, None if case["mode"] == "loss" else torch.full((rows,), mean, device="cuda")
        if case["mode"] == "mixed":
            s["rest"] = rest
            masked = torch.rand(rows, vocab, generator=g, device="cuda") < 0.1
            s["scores"].masked_fill_(masked.scatter_(1, s["index"].long(), False), -math.inf)  # what the teacher lists is not masked
            short = torch.randint(0, k + 1, (rows, 1), generator=g, device="cuda")
            s["index"].masked_fill_(torch.arange(k, device="cuda") >= torch.where(torch.rand(rows, 1, generator=g, device="cuda") < 0.25, short, k), -1)
            s["weight"] *= (torch.rand(rows, generator=g, device="cuda") < 0.9)  # padded positions have none
            if rows > 2:
                s["scores"][rows // 2] = -math.inf
        s["loss"] = torch.empty(rows, device="cuda")
        s["grad"] = None if case["mode"] == "loss" else torch.empty_like(s["scores"])
    return s


# ------------------------------------------------------------- plain forms


def _plain_quantise(x, kind, block):
    dtype, top = _F8[kind]
    rows, cols = x.shape
    full = x.new_zeros(-(-rows // block) * block, _blocks(cols) * 128, dtype=torch.float32)
    full[:rows, :cols] = x
    cut = full.view(-1, block, _blocks(cols), 128)
    t = cut.abs().amax((1, 3), keepdim=True)
    q = (cut * torch.where(t > 0, top / t, 0.0)).to(dtype)
    return q.view(full.shape)[:rows, :cols], (t / top)[:, 0, :, 0]


def _spread_scale(scale, block, rows, cols):
    return scale.repeat_interleave(block, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def _plain_product(a, a_scale, b, b_scale, block, bias, dtype):
    a = a.float() * _spread_scale(a_scale, 1, *a.shape)
    b = b.float() * _spread_scale(b_scale, block, *b.shape)
    out = a @ b.t()
    return (out if bias is None else out + bias).to(dtype)


def _log_shares(x, temperature):
    """Logarithms of softmax(x / T) over the last axis; -infinity throughout where nothing is left."""
    x = x.float()
    top = x.amax(-1, keepdim=True)
    z = (x - torch.where(top == -math.inf, 0.0, top)) / temperature
    return z - torch.log(torch.exp(z).sum(-1, keepdim=True, dtype=torch.float64)).float().clamp_min(-1.0)


def _plain_verify(target, draft, tokens, u, temperature, count):
    seqs, places, vocab = target.shape
    drafts = places - 1
    warm = temperature > 0
    t = torch.where(warm, temperature, 1.0)
    x = tokens.long()
    count = torch.full((seqs,), drafts, device=x.device) if count is None else count.long().clamp(0, drafts)
    best = target.float().argmax(-1)  # the lowest index among equal ones
    logp = _log_shares(target, t[:, None, None])
    p = logp[:, :drafts].gather(2, x[..., None])[..., 0]
    q = torch.zeros_like(p) if draft is None else _log_shares(draft, t[:, None, None]).gather(2, x[..., None])[..., 0]
    fits = torch.where(warm[:, None], u[:, :drafts] * torch.exp(q - p) < 1, best[:, :drafts] == x)
    fits &= (p > -math.inf) & (torch.arange(drafts, device=x.device) < count[:, None])
    accepted = fits.long().cumprod(1).sum(1)
    # the answer after them, in 64 bits: its border lies between running sums
    at = accepted[:, None, None]
    row = target.gather(1, at.expand(-1, 1, vocab))[:, 0].double()
    full = row.amax(1, keepdim=True) > -math.inf
    w = torch.exp(torch.where(full, row - row.amax(1, keepdim=True), -math.inf) / t[:, None].double())
    w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    late = (accepted < count)[:, None]
    if drafts > 0:
        at = at.clamp_max(drafts - 1)
        if draft is None:
            less = torch.zeros_like(w).scatter_(1, x.gather(1, at[..., 0]), 1.0)
        else:
            less = draft.gather(1, at.expand(-1, 1, vocab))[:, 0].double()
            less = torch.exp((less - less.amax(1, keepdim=True)) / t[:, None].double())
            less = less / less.sum(1, keepdim=True)
        rest = (w - less).clamp_min(0.0)
        w = torch.where(late & (rest.sum(1, keepdim=True) > 0), rest, w)
    upto = w.cumsum(1)
    part = torch.floor(u[:, drafts:].double() * 2.0 ** 30) * 2.0 ** -30
    last = (upto <= upto[:, -1:] * part).sum(1).clamp_max(vocab - 1)
    last = torch.where(warm, last, best.gather(1, accepted[:, None])[:, 0])
    last = torch.where(full[:, 0], last, -1)
    place = torch.arange(places, device=x.device)
    token = torch.where(place < accepted[:, None], torch.cat([x, x.new_zeros(seqs, 1)], 1), -1).scatter(1, accepted[:, None], last[:, None])
    logprob = torch.where(warm[:, None], logp.gather(2, token.clamp_min(0)[..., None])[..., 0], 0.0)
    return token.int(), accepted.int(), torch.where(token < 0, -math.inf, logprob)


def _plain_distill(scores, index, teacher, rest, weight, temperature, with_grad):
    z = scores.float() / temperature
    rows, vocab = z.shape
    there = (index >= 0) & (index < vocab)
    at = torch.where(there, index, 0).long()
    none = z.new_full((rows, 1), -math.inf)
    tau = torch.cat([torch.where(there, teacher.float() / temperature, -math.inf), none if rest is None else rest[:, None]], 1)

    def log_sum(v):
        top = v.amax(1, keepdim=True)
        base = torch.where(top == -math.inf, 0.0, top)
        return base + torch.log(torch.exp(v - base).sum(1, keepdim=True, dtype=torch.float64))  # 64 bits: a loss is a small difference of these

    all_t, all_z = log_sum(tau), log_sum(z)
    live = (all_t > -math.inf) & (all_z > -math.inf)
    if weight is not None:
        live &= weight[:, None] != 0
    scale = torch.where(live, z.new_ones(rows, 1) if weight is None else weight[:, None], 0.0)
    logp = torch.where(live, tau - all_t, -math.inf)
    p = torch.exp(logp)  # of a row's k entries, in 64 bits too
    listed_here = torch.zeros(rows, vocab + 1, dtype=torch.bool, device=z.device).scatter_(1, torch.where(there, at, vocab), True)[:, :vocab]
    others = z.masked_fill(listed_here, -math.inf)
    all_others = log_sum(others)
    logq = torch.cat([z.gather(1, at), all_others], 1) - all_z
    loss = (torch.where(p > 0, p * (logp - logq), 0.0).sum(1) * scale[:, 0] * temperature * temperature).float()
    if not with_grad:
        return loss, None
    share = torch.exp(others - torch.where(all_others == -math.inf, 0.0, all_others).float()) * (torch.exp(logq[:, -1:]) - p[:, -1:]).float()
    grad = torch.where(listed_here, torch.exp(z - all_z.float()), share)
    grad.scatter_add_(1, at, torch.where(there, -p[:, :-1], 0.0).float())
    return loss, torch.where(live, grad * (scale * temperature), 0.0).to(scores.dtype)


def run(s):
    if s["op"] == "quantise":
        if own:
            s["ops"].quantize_f8_dev(s["x"], s["q"], s["scale"], block_rows=s["block"])
            q, scale = s["q"], s["scale"]
        else:
            q, scale = _plain_quantise(s["x"], s["f8"], s["block"])
        return {"values": q.to(torch.bfloat16), "scale": scale}  # bf16 holds every 8-bit number
    if s["op"] == "product":
        if own:
            s["ops"].matmul_f8_dev(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"], bias=s["bias"])
            return s["out"]
        return _plain_product(s["a"], s["a_scale"], s["b"], s["b_scale"], s["block"], s["bias"], s["out"].dtype)
    if s["op"] == "verify":
        if own:
            s["ops"].verify_dev(s["target"], s["tokens"], s["u"], s["token"], s["accepted"], d_logprob=s["logprob"], d_draft=s["draft"],
                                draft_count=s["count"], temperature=s["temperature"])
            return {"token": s["token"], "accepted": s["accepted"], "logprob": s["logprob"]}
        token, accepted, logprob = _plain_verify(s["target"], s["draft"], s["tokens"], s["u"], s["temperature"], s["count"])
        return {"token": token, "accepted": accepted, "logprob": logprob}
    if own:
        s["ops"].distill_dev(s["scores"], s["index"], s["teacher"], d_loss=s["loss"], d_grad=s["grad"], rest=s["rest"], weight=s["weight"],
                             temperature=s["temperature"])
        return {"loss": s["loss"], "grad": s["grad"]}
    loss, grad = _plain_distill(s["scores"], s["index"], s["teacher"], s["rest"], s["weight"], s["temperature"], s["grad"] is not None)
    return {"loss": loss, "grad": grad}


# -------------------------------------------------------------- in 64 bits


def _exact_quantise(s):
    dtype, top = _F8[s["f8"]]
    bits, low = (3, -6) if s["f8"] == "e4m3" else (2, -14)  # of the mantissa, and the lowest normal exponent
    x, block = s["x"].double(), s["block"]
    rows, cols = x.shape
    values, scale = torch.empty_like(x), torch.empty(s["scale"].shape, dtype=torch.float64, device="cuda")
    for c in range(scale.shape[1]):
        part = x[:, 128 * c:128 * c + 128]
        row_top = part.abs().amax(1)
        t = torch.stack([v.amax() for v in row_top.split(block)]) if block > 1 else row_top
        scale[:, c] = t / top
        y = part * (top / t).repeat_interleave(block)[:rows, None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(1e-300))).clamp_min(low) - bits)
        values[:, 128 * c:128 * c + 128] = torch.round(y / step) * step
    return {"values": values, "scale": scale}


def _exact_product(s):
    m, n, k = s["m"], s["n"], s["k"]
    col = torch.arange(k, device="cuda") // 128
    a = s["a"].double() * s["a_scale"].double()[:, col]
    out = torch.empty(m, n, dtype=torch.float64, device="cuda")
    for j in range(0, n, 1 << 16):
        e = min(n, j + (1 << 16))
        row = torch.arange(j, e, device="cuda") // s["block"]
        out[:, j:e] = torch.mm(a, (s["b"][j:e].double() * s["b_scale"].double()[row][:, col]).t())
    return out if s["bias"] is None else out.add_(s["bias"].double())


def _exact_verify(s):
    seqs, drafts = s["seqs"], s["drafts"]
    token = torch.full((seqs, drafts + 1), -1, dtype=torch.int32)
    logprob = torch.full((seqs, drafts + 1), -math.inf, dtype=torch.float64)
    accepted = torch.zeros(seqs, dtype=torch.int32)
    for b in range(seqs):
        heat = float(s["temperature"][b])
        count = drafts if s["count"] is None else int(s["count"][b])
        for i in range(count + 1):
            row = s["target"][b, i].double()
            empty = bool(torch.isneginf(row).all())
            if empty:
                p = torch.zeros_like(row)
            elif heat > 0:
                p = torch.softmax(row / heat, 0)
            else:
                p = torch.zeros_like(row)
                p[int(torch.nonzero(row == row.max())[0])] = 1.0
            if i < count:
                x = int(s["tokens"][b, i])
                if s["draft"] is None or heat <= 0:
                    q = torch.zeros_like(row)
                    q[x] = 1.0
                else:
                    q = torch.softmax(s["draft"][b, i].double() / heat, 0)
                if (float(s["u"][b, i]) * float(q[x]) < float(p[x])) if heat > 0 else bool(p[x] > 0):
                    token[b, i], logprob[b, i] = x, math.log(float(p[x]))
                    accepted[b] += 1
                    continue
                left = (p - q).clamp_min(0) if heat > 0 else p
                left = left if float(left.sum()) > 0 else p
            else:
                left = p
            if not empty:
                passed = torch.nonzero(left.cumsum(0) > float(s["u"][b, drafts]) * left.sum())
                x = int(passed[0]) if len(passed) else int(torch.nonzero(left)[-1])
                token[b, i], logprob[b, i] = x, math.log(float(p[x]))
            break
    return {"token": token.cuda(), "accepted": accepted.cuda(), "logprob": logprob.cuda()}


def _exact_distill(s):
    rows, vocab, heat = s["rows"], s["vocab"], s["temperature"]
    loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    grad = None if s["grad"] is None else torch.zeros(rows, vocab, dtype=torch.float64, device="cuda")
    for r in range(0, rows, 256):
        e = min(rows, r + 256)
        for i in ([] if s["mode"] != "mixed" else range(r, e)):
            w = 1.0 if s["weight"] is None else float(s["weight"][i])
            have = s["index"][i] >= 0
            at = s["index"][i][have].long()
            z = s["scores"][i].double() / heat
            if w == 0 or bool(torch.isneginf(z).all()):
                continue
            p = torch.softmax(torch.cat([s["teacher"][i][have].double() / heat, s["rest"][i:i + 1].double()]), 0)
            q = torch.softmax(z, 0)
            outside = torch.ones(vocab, dtype=torch.bool, device="cuda")
            outside[at] = False
            z_rest = torch.logsumexp(z[outside], 0) - torch.logsumexp(z, 0)
            logq = torch.cat([torch.log_softmax(z, 0)[at], z_rest[None]])
            loss[i] = w * heat * heat * torch.xlogy(p, p).sub(torch.where(p > 0, p * logq, 0.0)).sum()
            d = q.clone()
            d[outside] = torch.softmax(z[outside], 0) * (torch.exp(z_rest) - p[-1])
            d[at] -= p[:-1]
            grad[i] = w * heat * d
        if s["mode"] != "mixed":
            w = torch.ones(e - r, 1, dtype=torch.float64, device="cuda") if s["weight"] is None else s["weight"][r:e, None].double()
            at = s["index"][r:e].long()
            logp = torch.log_softmax(s["teacher"][r:e].double() / heat, 1)
            logq = torch.log_softmax(s["scores"][r:e].double() / heat, 1)
            loss[r:e] = (w * heat * heat * (logp.exp() * (logp - logq.gather(1, at))).sum(1, keepdim=True))[:, 0]
            if grad is not None:
                grad[r:e] = w * heat * logq.exp().scatter_add_(1, at, -logp.exp())
    return {"loss": loss, "grad": grad}


def exact(case, seed):
    s = prepare(case, seed)
    return {"quantise": _exact_quantise, "product": _exact_product, "verify": _exact_verify, "distill": _exact_distill}[case["op"]](s)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "quantise":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": rows * cols * (size + 1) + 4 * -(-rows // case["block"]) * _blocks(cols), "flops": 3 * rows * cols}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        scales = 4 * _blocks(k) * (m + -(-n // case["block"]))
        return {"bytes": (m + n) * k + scales + m * n * size + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if case["op"] == "verify":
        rows = case["seqs"] * (case["drafts"] + 1 + (0 if case["mode"] == "none" else case["drafts"]))
        return {"bytes": rows * case["vocab"] * size + case["seqs"] * (case["drafts"] + 1) * 16, "flops": 4 * rows * case["vocab"]}
    rows, vocab, grad = case["rows"], case["vocab"], case["mode"] != "loss"
    return {"bytes": rows * (vocab * size * (2 if grad else 1) + case["k"] * (size + 4) + 12), "flops": rows * vocab * (8 if grad else 4)}
