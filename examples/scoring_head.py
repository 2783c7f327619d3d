"""A scoring head on 8-bit weights: rows quantised once, then per step the scores of a batch and one index drawn from
each.

The same three calls serve a vocabulary (hidden states in, next tokens out) and a corpus (query embeddings in, one
document drawn in proportion to its softmax weight): the weights are the rows that are scored, one scale a row.

    python examples/scoring_head.py --rows 32000 --depth 1024 --batch 16 --steps 32
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import resident_brute_force_gb300 as rbf  # noqa: E402


class ScoringHead:
    """Rows [n, depth] held in 8 bits; ``draw`` scores a batch against all of them and draws one row for each."""

    def __init__(self, rows: torch.Tensor, max_batch: int, stream=None):
        n, depth = rows.shape
        self.ops = rbf.Ops(max_batch, depth, stream=stream or torch.cuda.current_stream())
        pitch = -(-depth // 16) * 16  # rows on 16-byte boundaries
        self.weights = torch.empty(n, pitch, dtype=torch.int8, device=rows.device)[:, :depth]
        self.scale = torch.empty(n, device=rows.device)
        self.ops.quantize_rows_i8_dev(rows, self.weights, self.scale)
        self.scores = torch.empty(max_batch, -(-n // 8) * 8, dtype=torch.bfloat16, device=rows.device)[:, :n]
        self.index = torch.empty(max_batch, dtype=torch.int32, device=rows.device)
        self.logprob = torch.empty(max_batch, device=rows.device)

    def draw(self, x: torch.Tensor, u: torch.Tensor, **ask):
        """One index and its log-probability for each row of x [batch, depth]; u: random numbers in [0, 1); ask:
        temperature, top_k, top_p, min_p (see ``Ops.sample_dev``). The results are overwritten by the next call."""
        b = x.shape[0]
        scores, index, logprob = self.scores[:b], self.index[:b], self.logprob[:b]
        self.ops.linear_i8_dev(x, self.weights, self.scale, scores)
        self.ops.sample_dev(scores, u, index, logprob, **ask)
        return index, logprob


def main(argv=None) -> list[list[int]]:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--rows", type=int, default=32000)
    p.add_argument("--depth", type=int, default=1024)
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--seed", type=int, default=1)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(a.seed)
    rows = torch.randn(a.rows, a.depth, generator=g, device="cuda", dtype=torch.bfloat16)
    head = ScoringHead(rows, a.batch)
    ones = torch.ones(a.batch, device="cuda")
    ask = dict(temperature=0.8 * ones, top_k=torch.full((a.batch,), 50, dtype=torch.int32, device="cuda"), top_p=0.9 * ones)
    x = torch.randn(a.batch, a.depth, generator=g, device="cuda", dtype=torch.bfloat16) / a.depth ** 0.5
    drawn, begin, end = [], torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(a.steps + 1):
        if step == 1:  # the first step loads the kernels
            begin.record()
        index, _ = head.draw(x, torch.rand(a.batch, generator=g, device="cuda"), **ask)
        drawn.append(index.clone())
        x = rows[index.long()] / a.depth ** 0.5  # the drawn rows are the next step's inputs
    end.record()
    torch.cuda.synchronize()
    if head.ops.check_device_error() != rbf.RBF_OK:
        raise RuntimeError("a kernel reported a timeout")
    print(f"{a.steps} steps of {a.batch} x {a.rows} x {a.depth}: {1e3 * begin.elapsed_time(end) / a.steps:.1f} us a step")
    return torch.stack(drawn).tolist()


if __name__ == "__main__":
    main()
