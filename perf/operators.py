"""The scoring-head operators as measured cases: 8-bit row quantisation, the 8-bit integer product with a scale
for each token and channel, both in one call (a linear layer on 8-bit weights), and sampling from the scores.

`run` computes a case in its plain form (elementary torch operations) or, where `own` is true, with the calls a
user makes of this package. The sizes are those of this repository's corpora and batches (10k, 100k and 1M rows of
384 to 1024 values, batches of 1 to 256, wider layers for ingest) with odd and ragged ones among them.

What the operators compute:

  quantise   scale[i] = max_j |x[i, j]| / 127,  q[i, j] = rint(x[i, j] * (127 / max_j |x[i, j]|))
  product    out[i, j] = a_scale[i] * b_scale[j] * sum_k a[i, k] b[j, k]  (+ bias[j])
  linear     the product of quantise(x) with 8-bit weights
  sample     weights e = 2^((x - max x) log2(e) / temperature), held as whole multiples of 2^-36; the top_k largest are
             kept (equal scores: lowest index first), of those the fewest whose weights reach top_p of their sum, of
             those the ones with at least min_p of the largest weight (the largest one always); the token is the first
             one, in index order, at which the running sum of the kept weights passes u times their total
"""
import math

import torch

own = False

_FLOAT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_LOG2E = 1.4426950408889634
_ONE = 1 << 36  # fixed point: the largest weight of a row
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
        {"name": "quantise 1x768", "op": "quantise", "rows": 1, "cols": 768, "dtype": "f32"},
        # a corpus block at ingest
        {"name": "quantise 16384x8192", "op": "quantise", "rows": 16384, "cols": 8192, "dtype": "bf16"},
        # one query against a small 8-bit corpus: every score
        {"name": "product 1x10000x384", "op": "product", "m": 1, "n": 10000, "k": 384, "dtype": "f32", "bias": False},
        # one token against a 1M-row corpus: the weights are read once
        {"name": "product 1x1000000x768", "op": "product", "m": 1, "n": 1000000, "k": 768, "dtype": "f32", "bias": False},
        # a ragged batch on a ragged vocabulary
        {"name": "product 37x10007x1000", "op": "product", "m": 37, "n": 10007, "k": 1000, "dtype": "f16", "bias": True},
        # the full batch of queries against the 1M-row corpus
        {"name": "product 256x1000000x768", "op": "product", "m": 256, "n": 1000000, "k": 768, "dtype": "bf16", "bias": False},
        # decoding: a few tokens through a wide layer
        {"name": "linear 8x32000x4096", "op": "linear", "m": 8, "n": 32000, "k": 4096, "dtype": "bf16", "bias": False},
        # many tokens at once (ingest, or a prompt)
        {"name": "linear 4096x8192x4096", "op": "linear", "m": 4096, "n": 8192, "k": 4096, "dtype": "bf16", "bias": True},
        # one row of scores, the usual top-k and top-p together
        {"name": "sample 1x10000", "op": "sample", "rows": 1, "vocab": 10000, "dtype": "f32", "mode": "top_k_p"},
        # a ragged batch in which every row asks for something else; a masked-out row among them
        {"name": "sample 61x100003", "op": "sample", "rows": 61, "vocab": 100003, "dtype": "bf16", "mode": "mixed"},
        # the full batch on a large vocabulary, top-p alone
        {"name": "sample 256x128000", "op": "sample", "rows": 256, "vocab": 128000, "dtype": "bf16", "mode": "top_p"},
        # candidates drawn from the scores of a whole corpus
        {"name": "sample 8x1000000", "op": "sample", "rows": 8, "vocab": 1000000, "dtype": "f32", "mode": "min_p"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "linear", "sample", "sample"])
    if op == "quantise":
        rows, cols = _spread(rng, 1, 16384), _spread(rng, 16, 8192)
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["f32", "bf16", "f16"]) if rows * cols < 1 << 26 else "bf16"}
    if op == "sample":
        rows = _spread(rng, 1, 256)
        vocab = _spread(rng, 64, min(1000000, 32768000 // rows))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": rng.choice(["f32", "bf16", "f16"]) if rows * vocab < 16 << 20 else "bf16",
                "mode": rng.choice(["plain", "top_k", "top_p", "min_p", "top_k_p", "mixed"])}
    m, k = _spread(rng, 1, 4096), _spread(rng, 64, 8192)
    n = _spread(rng, 64, max(64, min(1000000, 768000000 // k, 256000000 // m, (1 << 37) // (m * k))))
    return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["f32", "bf16", "f16"]) if m * n < 1 << 26 else "bf16", "bias": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs


def _pitched(rows, cols, dtype, device="cuda"):
    """[rows, cols] in rows whose start is a multiple of 16 bytes, as the resident corpora are laid out."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // per) * per, dtype=dtype, device=device)[:, :cols]


def _embeddings(g, rows, cols, dtype):
    """Values with a few dominant directions and rows of different size, as embeddings and activations have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    x *= torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
    out = _pitched(rows, cols, dtype)
    out.copy_(x)
    return out


def _quantised(g, rows, cols):
    """8-bit rows with their scales, as the quantised corpus or layer has them."""
    q = _pitched(rows, cols, torch.int8)
    for r in range(0, rows, 1 << 17):  # a block at a time: the values before rounding are not all held at once
        n = min(1 << 17, rows - r)
        q[r:r + n].copy_((torch.randn(n, cols, generator=g, device="cuda") * 33.0).clamp_(-127, 127).round_())
    return q, torch.exp(0.3 * torch.randn(rows, generator=g, device="cuda")) * 0.001


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if own:
        s["ops"] = _ops()
    if case["op"] == "quantise":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _embeddings(g, rows, cols, _FLOAT[case["dtype"]])
        s["q"], s["scale"], s["values"] = _pitched(rows, cols, torch.int8), torch.empty(rows, device="cuda"), torch.empty_like(s["x"])
    elif case["op"] in ("product", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        s["b"], s["b_scale"] = _quantised(g, n, k)
        s["bias"] = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        s["out"] = torch.empty(m, n, dtype=_FLOAT[case["dtype"]], device="cuda")
        if case["op"] == "product":
            s["a"], s["a_scale"] = _quantised(g, m, k)
        else:
            s["x"] = _embeddings(g, m, k, _FLOAT[case["dtype"]])
    else:
        rows, vocab, mode = case["rows"], case["vocab"], case["mode"]
        x = 2.5 * torch.randn(rows, vocab, generator=g, device="cuda")
        few = torch.randint(0, vocab, (rows, min(40, vocab)), generator=g, device="cuda")
        x.scatter_add_(1, few, 6.0 * torch.rand(few.shape, generator=g, device="cuda"))  # a few likely ones
        u = lambda lo, hi: lo + (hi - lo) * torch.rand(rows, generator=g, device="cuda")  # noqa: E731
        s["u"], s["temperature"] = u(0.0, 1.0), u(0.6, 1.3)
        kinds = torch.randint(0, 6, (rows,), generator=g, device="cuda")  # mixed: what each row asks for
        mixed = mode == "mixed"
        s["top_k"] = torch.randint(1, 101, (rows,), generator=g, device="cuda", dtype=torch.int32) if mode in ("top_k", "top_k_p", "mixed") else None
        s["top_p"] = u(0.8, 0.99) if mode in ("top_p", "top_k_p", "mixed") else None
        s["min_p"] = u(0.02, 0.2) if mode in ("min_p", "mixed") else None
        if mixed:
            s["temperature"] = torch.where(kinds == 0, torch.zeros_like(s["temperature"]), s["temperature"])  # greedy
            s["top_k"] = torch.where((kinds == 1) | (kinds == 4), s["top_k"], torch.zeros_like(s["top_k"]))
            s["top_p"] = torch.where((kinds == 2) | (kinds == 4), s["top_p"], torch.ones_like(s["top_p"]))
            s["min_p"] = torch.where((kinds == 3) | (kinds == 4), s["min_p"], torch.zeros_like(s["min_p"]))
            x[torch.rand(rows, vocab, generator=g, device="cuda") < 0.25] = -math.inf  # an output grammar's mask
            x[rows // 2] = -math.inf if rows > 2 else x[rows // 2]
        s["x"] = x.to(_FLOAT[case["dtype"]])
        s["token"], s["logprob"] = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    return s


# ------------------------------------------------------------- plain forms


def _plain_quantise(x):
    x = x.float()
    amax = x.abs().amax(1, keepdim=True)
    q = torch.round(x * torch.where(amax > 0, 127.0 / amax, 0.0))
    return q, amax[:, 0] / 127.0


def _plain_product(a, a_scale, b, b_scale, bias, dtype):
    out = (a.float() @ b.float().t()) * a_scale[:, None] * b_scale
    return (out if bias is None else out + bias).to(dtype)


def _share(total, part):
    """total * part / 2^30, rounded down, in whole numbers (total <= 2^56, part <= 2^30)."""
    return ((total >> 24) * part + (((total & 0xFFFFFF) * part) >> 24)) >> 6


def _plain_sample(x, u, temperature, top_k, top_p, min_p):
    rows, vocab = x.shape
    x = x.float()
    top = x.amax(1, keepdim=True)
    warm = temperature[:, None] > 0
    rate = (_LOG2E / torch.where(warm, temperature[:, None], 1.0)).clamp_min(torch.finfo(torch.float32).tiny)
    e = torch.exp2(torch.where(x == top, 0.0, (x - top) * rate))
    w = torch.round(e * _ONE).long()
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    rank = torch.arange(vocab, device=x.device)
    k = torch.full((rows, 1), vocab, device=x.device) if top_k is None else torch.where(top_k[:, None] > 0, top_k[:, None].long(), vocab)
    keep = rank < torch.where(warm, k, 1)
    ws = torch.where(keep, w.gather(1, order), 0)
    upto = ws.cumsum(1)
    if top_p is not None:
        part = torch.round(top_p[:, None].clamp(0, 1) * 2.0 ** 30).long()
        keep &= upto - ws < _share(upto[:, -1:], part)
    if min_p is not None:
        keep &= e.gather(1, order) >= min_p[:, None]
    keep |= rank == 0
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0))
    upto = w.cumsum(1)
    total = upto[:, -1:]
    part = torch.floor(u[:, None] * 2.0 ** 30).long().clamp_(0, (1 << 30) - 1)
    token = (upto <= _share(total, part)).sum(1).clamp_max_(vocab - 1)
    w, total = w.gather(1, token[:, None])[:, 0], total[:, 0]
    logprob = torch.where(2 * w < total, torch.log(w.float() / total.float()), torch.log1p(-((total - w).float() / total.float())))
    none = top[:, 0] == -math.inf
    return torch.where(none, -1, token).int(), torch.where(none, -math.inf, logprob)


def run(s):
    if s["op"] == "quantise":
        if own:
            s["ops"].quantize_rows_i8_dev(s["x"], s["q"], s["scale"])
            torch.mul(s["q"], s["scale"][:, None], out=s["values"])  # what the 8-bit numbers stand for
            return {"values": s["values"], "scale": s["scale"]}
        q, scale = _plain_quantise(s["x"])
        return {"values": (q * scale[:, None]).to(s["x"].dtype), "scale": scale}
    if s["op"] == "product":
        if own:
            s["ops"].matmul_i8_dev(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"], bias=s["bias"])
            return s["out"]
        return _plain_product(s["a"], s["a_scale"], s["b"], s["b_scale"], s["bias"], s["out"].dtype)
    if s["op"] == "linear":
        if own:
            s["ops"].linear_i8_dev(s["x"], s["b"], s["b_scale"], s["out"], bias=s["bias"])
            return s["out"]
        q, scale = _plain_quantise(s["x"])
        return _plain_product(q, scale, s["b"], s["b_scale"], s["bias"], s["out"].dtype)
    if own:
        s["ops"].sample_dev(s["x"], s["u"], s["token"], s["logprob"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return {"token": s["token"], "logprob": s["logprob"]}
    token, logprob = _plain_sample(s["x"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    return {"token": token, "logprob": logprob}


# -------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        x = s["x"].double()
        scale = x.abs().amax(1) / 127
        return {"values": torch.round(x / scale[:, None]) * scale[:, None], "scale": scale}
    if case["op"] in ("product", "linear"):
        if case["op"] == "product":
            a = s["a"].double() * s["a_scale"].double()[:, None]
        else:
            x = s["x"].double()
            a_scale = x.abs().amax(1, keepdim=True) / 127
            a = torch.round(x / a_scale) * a_scale
        out = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
        for j in range(0, case["n"], 1 << 16):
            b = s["b"][j:j + (1 << 16)].double() * s["b_scale"][j:j + (1 << 16)].double()[:, None]
            out[:, j:j + (1 << 16)] = torch.mm(a, b.t())
        return out if s["bias"] is None else out.add_(s["bias"].double())
    tokens, logprobs = [], []
    for i in range(case["rows"]):
        x = s["x"][i].double()
        if bool(torch.isneginf(x).all()):
            tokens.append(-1)
            logprobs.append(-math.inf)
            continue
        t = float(s["temperature"][i])
        ranked, order = torch.sort(x, descending=True, stable=True)
        k = int(s["top_k"][i]) if s["top_k"] is not None and int(s["top_k"][i]) > 0 else x.numel()
        k = 1 if t <= 0 else min(k, x.numel())
        p = torch.exp((ranked[:k] - ranked[0]) / (t if t > 0 else 1.0))
        n = k
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            n = min(n, 1 + int((torch.cumsum(p, 0) < float(s["top_p"][i]) * p.sum()).sum()))
        if s["min_p"] is not None:
            n = min(n, max(1, int((p >= float(s["min_p"][i])).sum())))
        chosen = torch.sort(order[:n])[0]
        p = torch.exp((x[chosen] - ranked[0]) / (t if t > 0 else 1.0))
        p /= p.sum()
        at = min(int((torch.cumsum(p, 0) <= float(s["u"][i])).sum()), n - 1)
        tokens.append(int(chosen[at]))
        logprobs.append(math.log(float(p[at])))
    return {"token": torch.tensor(tokens, dtype=torch.int32, device="cuda"), "logprob": torch.tensor(logprobs, dtype=torch.float64, device="cuda")}


def work(case):
    if case["op"] == "quantise":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["rows"] * (case["cols"] * (size + 1) + 4), "flops": 3 * case["rows"] * case["cols"]}
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 28), "flops": 4 * case["rows"] * case["vocab"]}
    m, n, k = case["m"], case["n"], case["k"]
    size = 4 if case["dtype"] == "f32" else 2
    a = m * (k * size if case["op"] == "linear" else k + 4)
    return {"bytes": a + n * (k + 4) + m * n * size + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
