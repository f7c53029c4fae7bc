"""GPU tests of the 16-bit linear's workspace: the schedule goes by the sizes
and the alignment, a workspace holds all of it or is not used, and the splits
run on another stream and in a graph."""

import ctypes

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import assert_within, linear16_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def operands(m, n, k, dtype, offset=0, seed=0):
    """x [m][k] and w [n][k], x `offset` elements past a 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)
    x = torch.empty(m * k + 8, dtype=dtype, device="cuda")[offset:offset + m * k].view(m, k)
    x.copy_(torch.randn(m, k, generator=g))
    return x, (torch.randn(n, k, generator=g) * k ** -0.5).to(dtype).cuda()


def named_for(x, w):
    """Bytes that the operands' own plan takes."""
    out = ctypes.c_size_t(0)
    bq.check(bq.lib.svdq_linear16_workspace_size_for(x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0), x.shape[0], w.shape[0],
                                                     x.shape[1], ctypes.byref(out)))
    return out.value


@pytest.mark.parametrize("m,n,k,offset", [(100, 256, 4096, 0), (40, 130, 2056, 0), (100, 131, 2049, 0), (100, 256, 4096, 3)])
def test_fewer_bytes_than_named_run_in_one_piece(m, n, k, offset):
    for dtype in (BF, HF):
        x, w = operands(m, n, k, dtype, offset)
        named = bq.linear16_workspace_size(m, n, k)
        own = named_for(x, w)
        assert named >= own >= 3 * m * n * 4   # fewer bytes would still hold fewer splits
        whole = bq.linear16(x, w, workspace=None)
        split = bq.linear16(x, w)
        big = torch.empty(8 * m * n * 4 + 65536, dtype=torch.uint8, device="cuda")
        for size, used in ((named, True), (own, True), (big.numel(), True), (0, False), (16, False), (2 * m * n * 4, False),
                           (own - 16, False)):
            big.fill_(0x42)
            assert torch.equal(split if used else whole, bq.linear16(x, w, workspace=big[:size]))
            assert bool((big != 0x42).any()) == used   # whether parts were written
        want, bound = linear16_reference(x, w, None, "none", None, None, None)
        assert_within(whole, want, bound, "whole")
        assert_within(split, want, bound, "split")


@pytest.mark.parametrize("m,n,k", [(1, 40, 8192), (16, 64, 15360), (32, 200, 4096)])
def test_few_misaligned_rows_get_their_workspace(m, n, k):
    """Up to 32 rows take a kernel without a split where they are aligned,
    and the split one where they are not."""
    x, w = operands(m, n, k, BF, offset=1)
    named = bq.linear16_workspace_size(m, n, k)
    assert named > 0
    got = bq.linear16(x, w)
    assert torch.equal(got, bq.linear16(x, w, workspace=torch.empty(named, dtype=torch.uint8, device="cuda")))
    want, bound = linear16_reference(x, w, None, "none", None, None, None)
    assert_within(got, want, bound, "misaligned")
    assert_within(bq.linear16(x, w, workspace=None), want, bound, "misaligned, whole")


@pytest.mark.parametrize("m,n,k", [(150, 64, 8192), (90, 131, 4097)])
def test_splits_on_another_stream_and_in_a_graph(m, n, k):
    x, w = operands(m, n, k, BF)
    assert named_for(x, w) > 0
    want = bq.linear16(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = bq.linear16(x, w)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = bq.linear16(x, w)
    keep = x.clone()
    for i in range(4):
        x.copy_(keep * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, bq.linear16(x, w))
