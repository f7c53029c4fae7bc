"""GPU parity of the attention over the paged 8-bit cache against a plain
64-bit reference on the same codes."""

import ctypes
import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import assert_within
from tests._reference_cache import PAGE, paged_reference, random_cache, starts, tables

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def plan(total, batch, width, hq, hk, d):
    out = (ctypes.c_int32 * 2)()
    bq.check(bq.lib.svdq_debug_attention_paged_plan(total, batch, width, hq, hk, d, out))
    return tuple(out)


def check(new, lens, hq, hk, d, dtype, causal=True, scale=None, packed=True, fused=0, workspace="auto", width=None, low=-6, high=2, spoil=True):
    print("attention_paged", new, lens, hq, hk, d, dtype, causal, scale, packed, width, flush=True)
    g = torch.Generator().manual_seed(sum(new) * 3 + sum(lens) + hq * d)
    total = sum(new)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table, pages = tables(lens, g, width=width)
    print("plan", plan(total, len(new), table.shape[1], hq, hk, d), flush=True)
    cache = random_cache(pages, hk, d, g, low, high)
    if spoil:   # places past a sequence's end hold NaN
        for b, n in enumerate(lens):
            if n % PAGE and n <= table.shape[1] * PAGE:
                page = int(table[b, n // PAGE])
                cache.k.view(torch.uint8)[page, :, n % PAGE:] = 0x7F
                for p in range(n % PAGE, PAGE):
                    cache.v.view(torch.uint8)[page, :, p // 4 % 4, :, p // 16 * 4 + p % 4] = 0xFF
    whole = torch.randn(total, hq * d + fused, generator=g).to(dtype).cuda()
    q = whole[:, :hq * d].unflatten(1, (hq, d))
    # scores of a few units: keys are up to 448 * 2^2
    scale = 2.0 ** -9 / d ** 0.5 if scale is None else scale
    o, lse = bq.attention_paged(q, cache, table, lengths, cu_seqlens_q=starts(new) if packed else None, causal=causal, scale=scale,
                                return_lse=True, workspace=workspace)
    torch.cuda.synchronize()
    want, want_lse, bound, bound_lse = paged_reference(q, cache, table, lengths, new, causal, scale)
    assert_within(o, want, bound, "o")
    assert_within(lse, want_lse, bound_lse, "lse")
    return o, lse, (q, cache, table, lengths)


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_head_dims(d, dtype):
    check([1, 1, 1, 1], [1, 64, 130, 77], 4, 2, d, dtype, packed=False)
    check([1, 1, 1], [1500, 64, 0], 4, 2, d, dtype, packed=False)
    check([3, 40, 1], [100, 40, 200], 4, 2, d, dtype)
    check([100, 1], [170, 90], 4, 2, d, dtype)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (8, 1), (16, 1), (17, 1), (33, 1), (6, 3), (20, 4), (12, 12), (32, 8)])
def test_heads(hq, hk):
    for new, lens in (([1, 1, 1], [65, 300, 1]), ([1, 1], [2000, 1100]), ([2, 5], [70, 1300]), ([90, 7], [200, 7])):
        check(new, lens, hq, hk, 64, BF)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 1024, 1025, 4096, 5000])
def test_lengths(length):
    check([1], [length], 8, 2, 128, BF, packed=False)
    check([min(length, 3)], [length], 4, 1, 64, HF)


@pytest.mark.parametrize("causal", [False, True])
def test_chunks(causal):
    for dtype, d in ((BF, 128), (HF, 64)):
        check([130, 1, 65, 0, 33], [200, 129, 65, 70, 400], 4, 2, d, dtype, causal=causal)
        check([257], [700], 8, 1, d, dtype, causal=causal)
        check([64, 64], [64, 1000], 6, 6, d, dtype, causal=causal)


# sizes that tiles of many rows take: (new, lens, heads_q, heads_k, head_dim, causal)
MANY = [
    ([700, 300], [1290, 365], 32, 8, 128, True), ([700, 300], [1300, 300], 32, 8, 128, False), ([1000], [1000], 32, 8, 64, True),
    ([1100, 129], [1281, 129], 32, 8, 80, True), ([913, 400], [912, 1000], 32, 8, 112, False), ([900, 77], [960, 78], 32, 8, 48, True),
    ([600, 1, 5, 0, 8, 300], [700, 1200, 5, 70, 64, 1], 32, 8, 128, True),      # single tokens, and more queries than keys, among them
    ([600, 1, 5, 0, 8, 300], [700, 1000, 5, 70, 64, 1], 32, 8, 64, True), ([700, 400], [700, 449], 32, 16, 96, True), ([1030], [1030], 32, 8, 16, True),
]


@pytest.mark.parametrize("case", MANY)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_many_rows(case, dtype):
    new, lens, hq, hk, d, causal = case
    check(new, lens, hq, hk, d, dtype, causal=causal)


def test_many_rows_exponents_and_scores():
    for low, high, scale in ((-40, 40, 2.0 ** -51), (20, 40, 2.0 ** -51), (-6, 0, 0.5), (-6, 0, 2.0 ** -20)):
        check([700, 300], [1290, 365], 32, 8, 128, BF, low=low, high=high, scale=scale)
        check([1000], [1000], 32, 8, 64, HF, low=low, high=high, scale=scale)


def test_many_rows_of_pages_that_are_not_there():
    g = torch.Generator().manual_seed(14)
    for d in (64, 128):
        cache = random_cache(24, 8, d, g)
        cache.k.view(torch.uint8)[0], cache.v.view(torch.uint8)[0] = 0x7F, 0x7F       # page 0 is nobody's
        table = torch.arange(1, 24, dtype=torch.int32).repeat(2)[:40].view(2, 20).cuda()
        table[0, 3], table[0, 19], table[1, 0], table[1, 7] = -1, 24, -(2 ** 31), 2 ** 31 - 1
        new, lens = [900, 150], [1250, 700]
        assert plan(1070, 2, 20, 32, 8, d)[0] > 32
        q = torch.randn(1070, 32, d, generator=g).to(BF).cuda()
        o, lse = bq.attention_paged(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_seqlens_q=starts(new) + 7,
                                    scale=2.0 ** -12, return_lse=True)
        want, want_lse, bound, bound_lse = paged_reference(q, cache, table, torch.tensor(lens), new, True, 2.0 ** -12, first=7)
        assert_within(o, want, bound, "o")
        assert_within(lse, want_lse, bound_lse, "lse")
        assert (o[:7] == 0).all() and (o[-13:] == 0).all() and (lse[:7] == -math.inf).all() and (lse[-13:] == -math.inf).all()
        for cu in ([0, 5000, -3], [-5, 10, 5], [0, 999, 0]):
            for lengths in ([-1, 2 ** 31 - 1], [0, 0], [2 ** 31 - 1, -2 ** 31]):
                bq.attention_paged(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                                   cu_seqlens_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()


def test_chunks_against_long_caches():
    # more than 32 rows a sequence, few tiles: equal shares of tiles of 32 rows
    for new, lens, hq, hk, d in (([40], [3000], 8, 2, 128), ([64, 20, 1], [2000, 20, 1500], 4, 2, 64)):
        assert plan(sum(new), len(new), max(-(-n // PAGE) for n in lens) + 2, hq, hk, d) == (32, 512)
        check(new, lens, hq, hk, d, BF)
        check(new, lens, hq, hk, d, HF, causal=False)
        check(new, lens, hq, hk, d, BF, workspace=None)


def test_shares():
    """Long caches of very different lengths, cut into equal shares, and without a workspace."""
    lens = [5000, 3, 0, 1, 2000, 64, 1900, 129]
    for dtype in (BF, HF):
        for hq, hk in ((8, 2), (4, 4), (20, 1)):
            a = check([1] * 8, lens, hq, hk, 128, dtype, packed=False)
            b = check([1] * 8, lens, hq, hk, 128, dtype, packed=False, workspace=None)
            check([2, 1, 1, 0, 3, 1, 1, 2], lens, hq, hk, 64, dtype)
    q, cache, table, lengths = a[2]
    n = bq.attention_paged_workspace_size(8, 8, table.shape[1], 20, 1, 128)
    assert n > 0
    space = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    scale = 2.0 ** -9 / 128 ** 0.5
    for ws, want in ((space, a), (space[:-16], b)):
        o, lse = bq.attention_paged(q, cache, table, lengths, scale=scale, return_lse=True, workspace=ws)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_more_tiles_than_shares():
    check([1] * 200, [(i * 53) % 300 for i in range(200)], 8, 4, 64, BF, packed=False)
    check([1] * 70, [1100 + (i * 53) % 300 for i in range(70)], 8, 4, 64, BF, packed=False)
    check([i % 3 for i in range(150)], [i % 3 + (i * 91) % 1200 for i in range(150)], 4, 2, 64, HF)


def test_wide_table():
    # a table far wider than the sequences
    check([1, 1], [100, 30], 8, 2, 128, BF, width=500)
    check([4, 4], [100, 30], 8, 2, 128, BF, width=500)


@pytest.mark.parametrize("low,high", [(-40, -30), (-40, 40), (20, 40), (-12, 12)])
def test_exponents(low, high):
    # keys of every size: the scores stay small through the scale
    for new, lens in (([1, 1], [400, 1300]), ([70], [500])):
        check(new, lens, 4, 2, 64, BF, low=low, high=high, scale=2.0 ** (-11 - high))
        check(new, lens, 4, 2, 64, HF, low=low, high=high, scale=2.0 ** (-11 - high))


def test_sharp_and_flat_scores():
    for scale in (2.0 ** -20, 2.0 ** -6, 0.5):
        check([1, 1], [700, 2000], 4, 2, 64, BF, scale=scale, high=0)
        check([100], [300], 4, 2, 64, HF, scale=scale, high=0)


def test_strided_queries_and_out():
    o, lse, (q, cache, table, lengths) = check([1, 70], [100, 200], 4, 2, 64, BF, fused=64)
    whole = torch.full((71, 6, 64), 5.0, dtype=BF, device="cuda")
    got = bq.attention_paged(q, cache, table, lengths, cu_seqlens_q=starts([1, 70]), scale=2.0 ** -12, out=whole[:, 1:5])
    assert got.data_ptr() == whole[:, 1:5].data_ptr() and torch.equal(got, o)
    assert (whole[:, [0, 5]] == 5).all()


def test_pages_that_are_not_there_and_padding():
    g = torch.Generator().manual_seed(4)
    cache = random_cache(12, 2, 64, g)
    cache.k.view(torch.uint8)[0] = 0x7F          # page 0 is nobody's
    cache.v.view(torch.uint8)[0] = 0x7F
    table = torch.tensor([[1, -1, 2, 3], [4, 12, 2 ** 31 - 1, -2 ** 31], [-1, -1, -1, -1], [5, 6, 7, 8]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([230, 150, 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    for new in ([1, 1, 1, 1], [100, 3, 80, 40]):
        q = torch.randn(sum(new) + 20, 4, 64, generator=g).to(BF).cuda()
        o, lse = bq.attention_paged(q, cache, table, lengths, cu_seqlens_q=starts(new) + 7, scale=2.0 ** -12, return_lse=True)
        want, want_lse, bound, bound_lse = paged_reference(q, cache, table, lengths, new, True, 2.0 ** -12, first=7)
        assert_within(o, want, bound, "o")
        assert_within(lse, want_lse, bound_lse, "lse")
        assert (o[:7] == 0).all() and (o[-13:] == 0).all() and (lse[:7] == -math.inf).all() and (lse[-13:] == -math.inf).all()
        # starts and lengths that are none: nothing leaves the tensors
        for cu in ([0, 500, -3, 9, 9], [-5, 10, 5, 2 ** 31 - 1, 0], [0, 99, 0, 99, 0]):
            for lens in ([-1, 2 ** 31 - 1, -2 ** 31, 5], [0, 0, 0, 0]):
                bq.attention_paged(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                   cu_seqlens_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()


def test_hidden_rows():
    # more queries than keys: the first see nothing
    for new, lens in (([5], [3]), ([100], [40]), ([3, 2], [0, 1200])):
        check(new, lens, 4, 2, 64, BF)


def test_lengths_past_the_table():
    # keys past the table are hidden; the tokens stand where the length says
    for new, lens, width in (([1, 1], [150, 129], 2), ([4, 2], [130, 128], 2), ([5], [1400], 21), ([100], [230], 3), ([40, 90], [150, 300], 3),
                             ([300], [500], 5)):
        check(new, lens, 4, 2, 64, BF, width=width)
        check(new, lens, 4, 2, 128, HF, width=width)


def test_far_pages():
    pages = 2 ** 31 // (2 * PAGE * 128) + 5
    cache = bq.KVCache.allocate(pages, 2, 128)
    g = torch.Generator().manual_seed(2)
    small = random_cache(3, 2, 128, g)
    ids = [pages - 1, pages - 4, 5]
    for name in ("k", "v"):
        getattr(cache, name).view(torch.uint8)[ids] = getattr(small, name).view(torch.uint8)
    cache.exponents[ids] = small.exponents
    q = torch.randn(1, 4, 128, generator=g).to(BF).cuda()
    n = torch.tensor([180], dtype=torch.int32, device="cuda")
    o = bq.attention_paged(q, cache, torch.tensor([ids], dtype=torch.int32, device="cuda"), n, scale=2.0 ** -12)
    assert torch.equal(o, bq.attention_paged(q, small, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), n, scale=2.0 ** -12))


def test_stream_graph_and_repeat():
    for new, lens in (([1, 1, 1], [3000, 10, 900]), ([1, 1], [100, 200]), ([100, 1], [300, 70])):
        o, lse, (q, cache, table, lengths) = check(new, lens, 8, 2, 128, BF)
        cu = starts(new)

        def call():
            return bq.attention_paged(q, cache, table, lengths, cu_seqlens_q=cu, scale=2.0 ** -9 / 128 ** 0.5)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = [call() for _ in range(3)]
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(x, o) for x in got)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            static = call()
        for i in range(4):
            q.mul_(1.1)
            lengths -= 1
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(static, call())


def test_refuses():
    cache = bq.KVCache.allocate(2, 2, 32)
    q, table, n = torch.zeros(1, 4, 32, dtype=BF, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), \
        torch.ones(1, dtype=torch.int32, device="cuda")
    ok = dict(q=q, cache=cache, block_table=table, lengths=n)
    for kw in (dict(q=q.float()), dict(q=q.cpu()), dict(block_table=table.long()), dict(lengths=n.cpu()), dict(cu_seqlens_q=n.long()), dict(q=None),
               dict(cache=bq.KVCache(cache.k, cache.v.view(torch.uint8), cache.exponents)), dict(workspace=3), dict(scale="x"), dict(out=q.half())):
        with pytest.raises(TypeError):
            bq.attention_paged(**{**ok, **kw})
    for kw in (dict(q=q[:, :, :16]), dict(lengths=torch.ones(2, dtype=torch.int32, device="cuda")), dict(cu_seqlens_q=starts([1, 0])),
               dict(q=torch.zeros(2, 4, 32, dtype=BF, device="cuda")), dict(out=q[:, :2]), dict(workspace="none")):
        with pytest.raises(ValueError):
            bq.attention_paged(**{**ok, **kw})
    for kw in (dict(q=torch.zeros(1, 3, 32, dtype=BF, device="cuda")), dict(scale=-1.0), dict(scale=math.nan),
               dict(q=torch.zeros(1, 4, 36, dtype=BF, device="cuda")[:, :, 1:33])):
        with pytest.raises(bq.SvdqError):
            bq.attention_paged(**{**ok, **kw})
    assert bq.attention_paged(q[:0], cache, table, n, cu_seqlens_q=starts([0])).shape == (0, 4, 32)
