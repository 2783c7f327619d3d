"""The scoring-head calls captured in a graph and replayed on other inputs give the eager calls' results bit for bit."""
import pytest
import torch

import resident_brute_force_gb300 as rbf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,depth", [(1, 384), (3, 1000), (40, 1000), (200, 520)])
def test_replayed_graph_equals_eager_calls(batch, depth):
    n = 5003
    g = torch.Generator(device="cuda")
    g.manual_seed(batch)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream), rbf.Ops(256, 1024, stream=stream) as o:
        pitch = -(-depth // 16) * 16
        rows = torch.empty(n, pitch, dtype=torch.int8, device="cuda")[:, :depth]
        scale = torch.empty(n, device="cuda")
        o.quantize_rows_i8_dev(torch.randn(n, depth, generator=g, device="cuda"), rows, scale)
        x = torch.zeros(batch, depth, device="cuda", dtype=torch.bfloat16)
        u = torch.zeros(batch, device="cuda")
        temp = torch.full((batch,), 0.7, device="cuda")
        top_k = torch.full((batch,), 60, dtype=torch.int32, device="cuda")
        top_p = torch.full((batch,), 0.9, device="cuda")
        scores = torch.empty(batch, -(-n // 8) * 8, dtype=torch.bfloat16, device="cuda")[:, :n]
        index = torch.empty(batch, dtype=torch.int32, device="cuda")
        logprob = torch.empty(batch, device="cuda")

        def step():
            o.linear_i8_dev(x, rows, scale, scores)
            o.sample_dev(scores, u, index, logprob, temperature=temp, top_k=top_k, top_p=top_p)

        def inputs(seed):
            g.manual_seed(seed)
            # Rows of different size: the sums that one stage can reach differ from step to step.
            x.copy_(torch.randn(batch, depth, generator=g, device="cuda") * (1.0 + seed) + (seed % 2) * 3.0)
            u.copy_(torch.rand(batch, generator=g, device="cuda"))

        inputs(0)
        step()  # loads the kernels
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for seed in range(1, 5):
            inputs(seed)
            graph.replay()
            got = scores.clone(), index.clone(), logprob.clone()
            for out in (scores, index, logprob):
                out.zero_()
            step()
            for a, b in zip(got, (scores, index, logprob)):
                assert torch.equal(a, b)
            graph.replay()  # after an eager call
            for a, b in zip(got, (scores, index, logprob)):
                assert torch.equal(a, b)
        assert o.check_device_error() == 0
