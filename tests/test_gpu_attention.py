"""GPU parity of the attention over packed sequences against a plain 64-bit
reference, element by element, at the lengths, head layouts, strides and
masks where it can go wrong."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import assert_within, attention_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def cu(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def inputs(lens_q, lens_k, hq, hk, d, dtype, seed, layout="dense", q_std=1.0):
    g = torch.Generator().manual_seed(seed)
    tq, tk = sum(lens_q), sum(lens_k)
    if layout == "fused":
        x = torch.randn(tq, (hq + 2 * hk) * d, generator=g).to(dtype).cuda()
        return (x[:, :hq * d].view(tq, hq, d), x[:, hq * d:(hq + hk) * d].view(tk, hk, d),
                x[:, (hq + hk) * d:].view(tk, hk, d))
    if layout == "heads":      # [heads][tokens][d], rows padded by 8
        def one(t, h):
            return torch.randn(h, t, d + 8, generator=g).to(dtype).cuda()[:, :, :d].transpose(0, 1)
        return one(tq, hq), one(tk, hk), one(tk, hk)
    return ((torch.randn(tq, hq, d, generator=g) * q_std).to(dtype).cuda(), torch.randn(tk, hk, d, generator=g).to(dtype).cuda(),
            torch.randn(tk, hk, d, generator=g).to(dtype).cuda())


def check(q, k, v, lens_q, lens_k, causal, what, scale=None, packed=True, **kw):
    sc = q.shape[2] ** -0.5 if scale is None else scale
    print(what, lens_q[:12], lens_k[:12], tuple(q.shape), tuple(k.shape), q.dtype, causal, flush=True)
    args = dict(cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k)) if packed else {}
    o, lse = bq.attention(q, k, v, causal=causal, scale=scale, return_lse=True, **args, **kw)
    torch.cuda.synchronize()
    want, want_lse, bo, bl = attention_reference(q, k, v, lens_q, lens_k, causal, sc)
    assert_within(o, want, bo, what + " o")
    assert_within(lse, want_lse, bl, what + " lse")
    return o, lse


# lengths around the tiles of 32, 64 and 256 rows and of 32 and 64 keys
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 63, 64, 65, 127, 129, 255, 257, 513])
def test_one_sequence(n, causal):
    for dtype, d in ((BF, 128), (HF, 64)):
        q, k, v = inputs([n], [n], 2, 2, d, dtype, n)
        check(q, k, v, [n], [n], causal, f"self {n}", packed=False)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("nq,nk", [(1, 300), (300, 1), (70, 200), (200, 70), (257, 64), (64, 257), (5, 1000), (300, 0), (3, 0)])
def test_different_lengths(nq, nk, causal):
    """Causal with more queries than keys leaves the first rows empty."""
    q, k, v = inputs([nq], [nk], 3, 1, 128, BF, nq + nk)
    check(q, k, v, [nq], [nk], causal, f"{nq} x {nk}", packed=False)


@pytest.mark.parametrize("layout", ["dense", "fused", "heads"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_packed(causal, layout):
    lens = [77, 0, 1, 333, 64, 0, 13, 256, 0]
    for dtype, d, hq, hk in ((BF, 128, 8, 2), (HF, 64, 6, 6), (HF, 128, 3, 1)):
        q, k, v = inputs(lens, lens, hq, hk, d, dtype, d + hq, layout)
        check(q, k, v, lens, lens, causal, f"packed {layout}")


@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 72, 80, 96, 104, 120])
def test_head_dims(d):
    lens = [70, 129]
    for layout in ("fused", "dense"):
        q, k, v = inputs(lens, lens, 4, 2, d, BF if d % 16 else HF, d, layout)
        check(q, k, v, lens, lens, True, f"head_dim {d}")
    q, k, v = inputs([1, 1], [700, 3], 4, 2, d, BF, d + 1)
    check(q, k, v, [1, 1], [700, 3], False, f"head_dim {d}, one token")


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 16, 40])
def test_groups(group):
    lens_q, lens_k = [40, 1, 9], [120, 50, 0]
    q, k, v = inputs(lens_q, lens_k, 2 * group, 2, 64, BF, group)
    check(q, k, v, lens_q, lens_k, True, f"group {group}")


@pytest.mark.parametrize("batch", [2, 64, 65, 130, 4200])
def test_many_sequences(batch):
    """The search for a workgroup's sequence, at one, two and three levels."""
    g = torch.Generator().manual_seed(batch)
    lens_q = torch.randint(0, 4, (batch,), generator=g).tolist()
    lens_k = torch.randint(0, 6, (batch,), generator=g).tolist()
    q, k, v = inputs(lens_q, lens_k, 2, 1, 16, HF, batch)
    check(q, k, v, lens_q, lens_k, True, f"batch {batch}")
    if batch < 200:
        lens = [40 * n for n in lens_q]
        q, k, v = inputs(lens, lens, 2, 1, 16, HF, batch)
        check(q, k, v, lens, lens, True, f"batch {batch}, longer")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_one_token_against_caches(dtype):
    """Few queries: the keys are cut into parts that a second kernel joins;
    without a workspace one workgroup runs through them."""
    lens_q, lens_k = [1, 1, 2, 1, 1, 0], [5000, 1, 2049, 0, 3333, 10]
    for hq, hk, d in ((8, 2, 128), (3, 3, 64)):
        assert bq.attention_workspace_size(sum(lens_q), sum(lens_k), 6, hq, hk, d) > 0
        q, k, v = inputs(lens_q, lens_k, hq, hk, d, dtype, hq)
        for causal in (False, True):
            a, la = check(q, k, v, lens_q, lens_k, causal, "split")
            b, lb = check(q, k, v, lens_q, lens_k, causal, "whole", workspace=None)
            again = bq.attention(q, k, v, cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k), causal=causal)
            assert torch.equal(a, again)


@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d", [
    ([1], [100000], 4, 1, 64),                        # one sequence over every workgroup
    ([1, 0, 3, 1], [0, 500, 20000, 64], 2, 2, 128),   # no keys, no queries, one long
    ([70, 1, 40], [900, 9000, 33], 3, 1, 40),         # several tiles of rows in a sequence
    ([1] * 100, [7 * (i % 9) if i % 10 else 3000 for i in range(100)], 1, 1, 64),   # parts that run over many sequences
    ([2, 1], [257, 4000], 16, 2, 128),
])
def test_equal_shares_of_the_keys(lens_q, lens_k, hq, hk, d):
    """Few rows and heads: parts of equal work, whose ends fall anywhere in
    the sequences, joined per row."""
    assert bq.attention_workspace_size(sum(lens_q), sum(lens_k), len(lens_q), hq, hk, d) > 0
    q, k, v = inputs(lens_q, lens_k, hq, hk, d, BF, 17)
    for causal in (False, True):
        a, la = check(q, k, v, lens_q, lens_k, causal, "shares")
        args = dict(cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k), causal=causal, return_lse=True)
        b, lb = bq.attention(q, k, v, **args)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d", [
    ([1, 2, 2, 1, 1], [1342, 1, 4, 124, 2100], 6, 6, 128),       # parts over several sequences, short ones among them
    ([1] * 40, [1, 0, 3, 40, 4000] * 8, 4, 2, 96),
    ([33, 0, 64, 1], [700, 50, 1, 2900], 2, 1, 64),              # tiles of rows of a few tiles of keys
    ([1], [1025], 1, 1, 8),
])
def test_shares_that_end_where_a_tile_of_rows_starts(lens_q, lens_k, hq, hk, d):
    assert bq.attention_workspace_size(sum(lens_q), sum(lens_k), len(lens_q), hq, hk, d) > 0
    for seed in (1, 2):
        q, k, v = inputs(lens_q, lens_k, hq, hk, d, HF, seed)
        for causal in (False, True):
            check(q, k, v, lens_q, lens_k, causal, "shares")
            check(q, k, v, lens_q, lens_k, causal, "whole", workspace=None)


def test_long_keys_and_few_heads():
    """One workgroup a CU at most: the keys are cut in two."""
    for lens_q, lens_k, hq, hk in (([4100], [4200], 4, 4), ([2100, 4001], [8000, 300], 2, 2)):
        q, k, v = inputs(lens_q, lens_k, hq, hk, 40, BF, 9)
        for causal in (False, True):
            check(q, k, v, lens_q, lens_k, causal, "cut in two")


@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d", [
    ([300, 20, 700, 0, 130], [1000, 0, 64, 2000, 1100], 2, 2, 128),    # parts of unequal numbers of tiles, of one and of none
    ([500, 300], [65, 3000], 3, 3, 64),
    ([1000], [771], 4, 1, 72),
    ([513], [4097], 2, 2, 128),                                         # and split over workgroups as well
])
def test_two_parts_of_the_keys(lens_q, lens_k, hq, hk, d):
    """A grid of few tiles of 128 rows with long keys: the waves of a
    workgroup take them in two parts."""
    for dtype in (BF, HF):
        q, k, v = inputs(lens_q, lens_k, hq, hk, d, dtype, 23)
        for causal in (False, True):
            a, la = check(q, k, v, lens_q, lens_k, causal, "parts")
            check(q, k, v, lens_q, lens_k, causal, "parts, whole", workspace=None)
            args = dict(cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k), causal=causal, return_lse=True)
            b, lb = bq.attention(q, k, v, **args)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_split_with_many_rows():
    """A grid of wide tiles that would leave the device idle is cut along the
    keys as well."""
    lens_q, lens_k = [200, 90], [3000, 2100]
    assert bq.attention_workspace_size(290, 5100, 2, 4, 1, 128) > 0
    q, k, v = inputs(lens_q, lens_k, 4, 1, 128, BF, 5)
    for causal in (False, True):
        check(q, k, v, lens_q, lens_k, causal, "split, many rows")
        check(q, k, v, lens_q, lens_k, causal, "whole, many rows", workspace=None)


@pytest.mark.parametrize("n", [40, 300])
def test_rising_and_extreme_scores(n):
    """Scores that rise along the keys make the reference move in every
    tile; large scores leave one weight; equal ones leave them all."""
    for dtype in (BF, HF):
        q, k, v = inputs([n], [n], 2, 2, 64, dtype, 3)
        k = (k.float() * 0.05 + torch.linspace(-3, 3, n, device="cuda")[:, None, None]).to(dtype)
        check(q.abs(), k, v, [n], [n], False, "rising", packed=False)
        check(q.abs(), k.flip(0).contiguous(), v, [n], [n], True, "falling", packed=False)
        check(q * 16, k, v, [n], [n], True, "large", scale=4.0, packed=False)
        check(torch.zeros_like(q), k, v, [n], [n], False, "equal", packed=False)


def test_what_a_row_cannot_see_does_not_reach_it():
    """NaN and infinities in other sequences, in keys hidden by the causal
    rule and past the end of a cache leave the rows as they are; a NaN in a
    query stays in its row."""
    lens = [50, 90, 33]
    q, k, v = inputs(lens, lens, 4, 2, 128, BF, 9)
    for few in (False, True):
        ql = [1, 1, 1] if few else lens
        qq = q[:3].contiguous() if few else q
        args = dict(cu_seqlens_q=cu(ql), cu_seqlens_k=cu(lens))
        clean = bq.attention(qq, k, v, **args)
        k2, v2 = k.clone(), v.clone()
        k2[50:140], v2[50:140] = math.nan, math.inf      # the middle sequence
        dirty = bq.attention(qq, k2, v2, **args)
        a, b = (1, 2) if few else (50, 140)
        assert torch.equal(clean[:a], dirty[:a]) and torch.equal(clean[b:], dirty[b:])
    # causal: a key is hidden from every query before it
    k2 = k.clone()
    k2[49] = math.nan
    args = dict(cu_seqlens_q=cu(lens), cu_seqlens_k=cu(lens), causal=True)
    clean, dirty = bq.attention(q, k, v, **args), bq.attention(q, k2, v, **args)
    assert torch.equal(clean[:49], dirty[:49]) and torch.equal(clean[50:], dirty[50:])
    assert dirty[49].isnan().all()
    q2 = q.clone()
    q2[7, 1] = math.nan
    dirty = bq.attention(q2, k, v, **args)
    assert dirty[7, 1].isnan().all()
    keep = torch.ones(sum(lens), 4, dtype=torch.bool, device="cuda")
    keep[7, 1] = False
    assert torch.equal(clean[keep], dirty[keep])
    # a cache longer than what is filled: the tail is never read
    cache_k, cache_v = torch.full((400, 2, 128), math.nan, dtype=BF, device="cuda"), torch.full((400, 2, 128), math.inf, dtype=BF, device="cuda")
    cache_k[:150], cache_v[:150] = k[:150], v[:150]
    starts = torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    for nq in (1, 100):
        at = torch.tensor([0, nq], dtype=torch.int32, device="cuda")
        got = bq.attention(q[:nq], cache_k, cache_v, cu_seqlens_q=at, cu_seqlens_k=starts)
        want, _, bound, _ = attention_reference(q[:nq], k[:150], v[:150], [nq], [150], False, 128 ** -0.5)
        assert_within(got, want, bound, "cache")


def test_long_cache_offsets_pass_32_bits():
    """A cache whose tokens lie 4 MB apart: offsets pass 2^32 bytes."""
    stride, n = 2 ** 21, 1300
    buf = torch.empty(stride * n + 512, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    k = buf.as_strided((n, 1, 128), (stride, 128, 1))
    v = buf[256:].as_strided((n, 1, 128), (stride, 128, 1))
    k.copy_(torch.randn(n, 1, 128, generator=g))
    v.copy_(torch.randn(n, 1, 128, generator=g))
    for nq in (1, 80):
        q = torch.randn(nq, 1, 128, generator=g).to(BF).cuda()
        check(q, k, v, [nq], [n], True, "far", packed=False)


def test_out_with_strides():
    lens = [30, 100]
    q, k, v = inputs(lens, lens, 2, 2, 80, HF, 4)
    whole = torch.full((130, 4, 88), 7.0, dtype=HF, device="cuda")
    out = whole[:, 1:3, :80]
    check(q, k, v, lens, lens, False, "strided out", out=out)
    assert (whole[:, 0] == 7).all() and (whole[:, 3] == 7).all() and (whole[:, :, 80:] == 7).all()


def test_nothing_to_do():
    q = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    k = torch.randn(5, 2, 64, device="cuda").to(BF)
    assert bq.attention(q, k, k).shape == (0, 4, 64)
    o, lse = bq.attention(k, k[:0], k[:0], return_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()


def test_another_stream_and_graph():
    lens_q, lens_k = [1, 1, 60], [900, 2000, 60]
    q, k, v = inputs(lens_q, lens_k, 4, 2, 128, BF, 11)
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
    for i in range(3):
        q.copy_(keep * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, bq.attention(q, k, v, **args))


def test_wrapper_refuses():
    q, k, v = inputs([8], [8], 4, 2, 64, BF, 1)
    c = cu([8])
    with pytest.raises(TypeError):
        bq.attention(q.float(), k.float(), v.float())
    with pytest.raises(TypeError):
        bq.attention(q, k.half(), v)
    with pytest.raises(TypeError):
        bq.attention(q.cpu(), k, v)
    with pytest.raises(ValueError):
        bq.attention(q, k, v[:, :1])
    with pytest.raises(ValueError):
        bq.attention(q, k, v, cu_seqlens_k=c)
    with pytest.raises(TypeError):
        bq.attention(q, k, v, cu_seqlens_q=c.long())
    with pytest.raises(ValueError):
        bq.attention(q, k, v, cu_seqlens_q=c, cu_seqlens_k=cu([4, 4]))
    with pytest.raises(bq.SvdqError):
        bq.attention(q[:, :3], k, v)                       # 3 heads over 2
    with pytest.raises(bq.SvdqError):
        bq.attention(q, k, v, scale=0.0)
    with pytest.raises(bq.SvdqError):
        bq.attention(q[..., :60], k[..., :60], v[..., :60])   # head_dim % 8
    with pytest.raises(bq.SvdqError):
        bq.attention(q[:, :, 1:57], k[:, :, 1:57], v[:, :, 1:57])   # misaligned
