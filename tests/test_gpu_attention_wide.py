"""GPU parity of attention's tiles of 256 rows (full attention over long keys
with many rows) against a plain 64-bit reference: row and key remainders,
sequences of few keys among long ones, heads that do not fill a tile."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._plans import attention_plan
from tests._reference16 import assert_within, attention_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def cu(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def check(q, k, v, lens_q, lens_k, what, **kw):
    print(what, lens_q, lens_k, tuple(q.shape), tuple(k.shape), q.dtype, flush=True)
    o, lse = bq.attention(q, k, v, cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k), return_lse=True, **kw)
    torch.cuda.synchronize()
    want, want_lse, bo, bl = attention_reference(q, k, v, lens_q, lens_k, False, q.shape[2] ** -0.5)
    assert_within(o, want, bo, what + " o")
    assert_within(lse, want_lse, bl, what + " lse")
    return o


def inputs(lens_q, lens_k, hq, hk, d, dtype, layout="dense"):
    g = torch.Generator().manual_seed(sum(lens_q) + d)
    tq, tk = sum(lens_q), sum(lens_k)

    def one(t, h):
        if layout == "heads":   # [heads][tokens][d], rows padded by 8
            return torch.randn(h, t, d + 8, generator=g).to(dtype).cuda()[:, :, :d].transpose(0, 1)
        return torch.randn(t, h, d, generator=g).to(dtype).cuda()

    return one(tq, hq), one(tk, hk), one(tk, hk)


CASES = [
    ([1100, 1301], [1100, 1301], 32, 32, 128),                      # remainders of rows and keys
    ([4225], [1029], 8, 8, 64),                                     # one row past a tile
    ([700, 0, 1, 1400, 300], [3000, 40, 5000, 1, 100], 16, 16, 72),   # no queries, one query, one key among long ones
    ([700, 0, 1, 1400, 300], [3000, 40, 5000, 1, 100], 32, 16, 128),
    ([300] * 7, [1, 64, 65, 128, 129, 192, 8000], 17, 17, 64),      # one to four tiles of keys: fewer than are loaded ahead
    ([300] * 8, [0, 192, 193, 256, 257, 320, 321, 9000], 17, 17, 128),
    ([2750], [2051], 36, 12, 40),                                   # three heads a key head
    ([1, 2000] + [40] * 69, [70000, 700] + [40] * 69, 10, 10, 24),   # more sequences than the lanes of a wave hold
]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d", CASES)
def test_tiles_of_256_rows(lens_q, lens_k, hq, hk, d, dtype):
    assert attention_plan(lens_q, lens_k, hq, hk, d, False) == (256, 1, 1, 0)
    q, k, v = inputs(lens_q, lens_k, hq, hk, d, dtype)
    a = check(q, k, v, lens_q, lens_k, "256 rows")
    b = bq.attention(q, k, v, cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k))
    assert torch.equal(a, b)


@pytest.mark.parametrize("d", [128, 64])
def test_strided_in_and_out(d):
    lens_q, lens_k, h = [1203, 900], [1500, 1001], 18
    assert attention_plan(lens_q, lens_k, h, h, d, False)[0] == 256
    q, k, v = inputs(lens_q, lens_k, h, h, d, BF, "heads")
    whole = torch.full((sum(lens_q), h + 2, d + 8), 7.0, dtype=BF, device="cuda")
    check(q, k, v, lens_q, lens_k, "strided", out=whole[:, 1:-1, :d])
    assert (whole[:, 0] == 7).all() and (whole[:, -1] == 7).all() and (whole[:, :, d:] == 7).all()


@pytest.mark.parametrize("d", [128, 64])
def test_rising_and_extreme_scores(d):
    n, h = 2100, 17
    assert attention_plan([n], [n], h, h, d, False)[0] == 256
    for dtype in (BF, HF):
        q, k, v = inputs([n], [n], h, h, d, dtype)
        k = (k.float() * 0.05 + torch.linspace(-3, 3, n, device="cuda")[:, None, None]).to(dtype)
        check(q.abs(), k, v, [n], [n], "rising")
        check(q.abs(), k.flip(0).contiguous(), v, [n], [n], "falling")
        check(q * 8, k, v, [n], [n], "large")


def test_other_sequences_and_what_is_past_the_keys():
    """NaN and infinities of another sequence and past the last key leave a
    sequence as it is."""
    lens_q, lens_k, h, d = [1203, 900, 400], [1500, 1001, 700], 16, 128
    assert attention_plan(lens_q, lens_k, h, h, d, False)[0] == 256
    q, k, v = inputs(lens_q, lens_k, h, h, d, BF)
    clean = bq.attention(q, k, v, cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k))
    k2, v2 = k.clone(), v.clone()
    k2[1500:2501], v2[1500:2501] = math.nan, math.inf
    dirty = bq.attention(q, k2, v2, cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k))
    assert torch.equal(clean[:1203], dirty[:1203]) and torch.equal(clean[2103:], dirty[2103:])
    assert dirty[1203:2103].isnan().all()
    ends = torch.tensor([0, 1500, 2501, 3100], dtype=torch.int32, device="cuda")   # the last cache is filled up to 599 keys
    k2, v2 = k.clone(), v.clone()
    k2[3100:], v2[3100:] = math.nan, math.inf
    got = bq.attention(q, k2, v2, cu_seqlens_q=cu(lens_q), cu_seqlens_k=ends)
    want, _, bound, _ = attention_reference(q, k[:3100], v[:3100], lens_q, [1500, 1001, 599], False, d ** -0.5)
    assert_within(got, want, bound, "filled in part")


@pytest.mark.parametrize("hq,nq", [(1, 33025), (4, 8300)])
def test_offsets_pass_32_bits(hq, nq):
    """Keys that lie 4 MB apart: offsets pass 2^32 bytes."""
    stride, n = 2 ** 21, 1029
    assert attention_plan([nq], [n], hq, 1, 128, False) == (256, 1, 1, 0)
    buf = torch.empty(stride * n + 512, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    k = buf.as_strided((n, 1, 128), (stride, 128, 1))
    v = buf[256:].as_strided((n, 1, 128), (stride, 128, 1))
    k.copy_(torch.randn(n, 1, 128, generator=g))
    v.copy_(torch.randn(n, 1, 128, generator=g))
    q = torch.randn(nq, hq, 128, generator=g).to(BF).cuda()
    check(q, k, v, [nq], [n], "far")


def test_equal_shares_on_another_stream_and_in_a_graph():
    """One token against long caches: the workspace and the joining kernel
    on another stream and in a graph, each replay checked."""
    lens_q, lens_k, hq, hk, d = [1, 1, 2], [5000, 1, 2049], 8, 2, 128
    assert attention_plan(lens_q, lens_k, hq, hk, d, True)[3] > 0 and bq.attention_workspace_size(4, 7050, 3, hq, hk, d) > 0
    q, k, v = inputs(lens_q, lens_k, hq, hk, d, BF)
    args = dict(cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k), causal=True)
    want = bq.attention(q, k, v, **args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = bq.attention(q, k, v, **args)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = bq.attention(q, k, v, **args)
    keep = q.clone()
    for i in range(4):
        q.copy_(keep * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, bq.attention(q, k, v, **args))
