"""The attention over the paged cache repeats itself bit by bit in every
schedule: call after call, on another stream and replayed from a graph, with
the program's own work between."""

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference_cache import starts
from tests.test_gpu_attention_paged import check, plan

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

# (new, lengths, heads_q, heads_k, head_dim, causal, schedule)
CASES = [
    ([700, 300], [1290, 365], 32, 8, 128, True, (256, 0)), ([700, 300], [1300, 300], 32, 8, 128, False, (256, 0)),
    ([600, 1, 5, 0, 8, 300], [700, 1200, 5, 70, 64, 300], 32, 8, 128, True, (256, 0)),
    ([1000], [1100], 32, 8, 64, True, (128, 0)), ([900, 77], [960, 78], 32, 8, 48, True, (128, 0)),
    ([40], [3000], 8, 2, 128, True, (32, 512)),
    # the schedules that smaller calls take
    ([1, 1, 1], [3000, 10, 900], 8, 2, 128, True, (16, 512)), ([1, 1], [100, 200], 8, 2, 128, True, (16, 0)),
    ([100, 1], [300, 70], 8, 2, 128, True, (32, 0)),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_repeat_stream_and_graph(case, dtype):
    new, lens, hq, hk, d, causal, schedule = case
    o, lse, (q, cache, table, lengths) = check(new, lens, hq, hk, d, dtype, causal=causal)
    assert plan(sum(new), len(new), table.shape[1], hq, hk, d) == schedule
    cu, scale = starts(new), 2.0 ** -9 / d ** 0.5

    def call():
        return bq.attention_paged(q, cache, table, lengths, cu_seqlens_q=cu, causal=causal, scale=scale, return_lse=True)

    def same(a, b):
        return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

    assert all(same(call(), (o, lse)) for _ in range(5))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [call() for _ in range(5)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(same(a, (o, lse)) for a in got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = call()
    for i in range(5):
        q.mul_(1.1)
        lengths -= 1
        graph.replay()
        torch.cuda.synchronize()
        assert same(static, call())
