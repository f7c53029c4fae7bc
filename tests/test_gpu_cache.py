"""GPU parity of appending to the paged 8-bit cache: every byte of the cache
and the rotated queries, against a plain 64-bit model of the page's rule."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import TINY, U16, assert_within
from tests._reference_cache import PAGE, Snapshot, check_append, random_cache, starts, tables, turned

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def check(new, old, hq, hk, d, dtype, rotary=None, interleaved=False, packed=True, fused=True, shift=0, in_place=False, std=1.0, cache=None,
          rope_rows=None):
    print("cache_append", new, old, hq, hk, d, dtype, rotary, interleaved, packed, fused, shift, flush=True)
    g = torch.Generator().manual_seed(sum(new) * 7 + sum(old) + d)
    total = sum(new)
    lengths = torch.tensor([a + b for a, b in zip(new, old)], dtype=torch.int32, device="cuda")
    table, pages = tables([a + b for a, b in zip(new, old)], g)
    cache = cache or random_cache(pages, hk, d, g)
    if fused:
        qkv = (torch.randn(total, (hq + 2 * hk) * d + shift, generator=g) * std).to(dtype).cuda()[:, shift:]
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([hq * d, hk * d, hk * d], dim=1))
    else:
        q, k, v = ((torch.randn(total, h, d, generator=g) * std).to(dtype).cuda() for h in (hq, hk, hk))
    rotary = d if rotary is None else rotary
    rope = bq.rope_table(rope_rows or int(lengths.max()) + 1, rotary) if rotary else None
    before, q_before = Snapshot(cache), q.clone()
    got = bq.cache_append(cache, k, v, table, lengths, q=q, rope=rope, cu_seqlens=starts(new) if packed else None,
                          interleaved=interleaved, q_out=q if in_place else None)
    torch.cuda.synchronize()
    check_append(before, cache, k, v, table, lengths, new, rope, interleaved)
    positions = torch.cat([torch.arange(b, a + b) for a, b in zip(new, old)])
    want, bound = turned(q_before, positions, rope, interleaved)
    assert_within(got, want, bound + U16[dtype] * (want.abs() + bound) + TINY[dtype], "q")
    return cache, table, lengths


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_head_dims(d, dtype):
    check([1, 1, 1, 1, 1], [0, 5, 63, 64, 127], 4, 2, d, dtype, packed=False)
    check([70, 0, 3, 64, 1], [30, 9, 61, 128, 0], 4, 2, d, dtype, interleaved=True)


@pytest.mark.parametrize("rotary", [0, 16, 32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations(rotary, interleaved):
    check([1, 1, 1], [100, 0, 1000], 8, 1, 128, BF, rotary=rotary, interleaved=interleaved, packed=False)
    check([100, 33], [63, 0], 3, 3, 128, HF, rotary=rotary, interleaved=interleaved, fused=False)
    check([100, 33], [63, 0], 3, 3, 128, BF, rotary=rotary, interleaved=interleaved, in_place=True)


@pytest.mark.parametrize("shift", [0, 1, 3])
def test_alignment(shift):
    check([5, 66], [62, 3], 4, 4, 64, BF, shift=shift)
    check([1, 1], [62, 3], 4, 4, 80, HF, shift=shift, packed=False, rotary=32)


def test_ragged_pack():
    new = [1024, 77, 513, 1, 333, 0, 150, 512, 13, 64]
    check(new, [0, 0, 640, 100, 31, 5, 0, 1000, 63, 64], 4, 2, 128, BF)


def test_many_sequences():
    # more sequences than a wave looks at at a time
    n = 150
    check([i % 3 for i in range(n)], [(i * 37) % 200 for i in range(n)], 2, 1, 64, BF)
    check([1] * n, [(i * 37) % 200 for i in range(n)], 2, 2, 64, HF, packed=False)
    check([0] * n + [200, 7], [0] * n + [10, 60], 2, 1, 64, BF)


def test_growing_exponents():
    """A sequence that grows token by token, some far larger than all before."""
    g = torch.Generator().manual_seed(5)
    for dtype in (BF, HF):
        cache, table = random_cache(4, 2, 64, g), torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
        for i in range(140):
            scale = 2.0 ** ((i * 5) % 13 - 6)
            k, v = ((torch.randn(1, 2, 64, generator=g) * scale).to(dtype).cuda() for _ in range(2))
            lengths = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
            before = Snapshot(cache)
            assert bq.cache_append(cache, k, v, table, lengths) is None
            check_append(before, cache, k, v, table, lengths, [1])


def test_same_as_at_once():
    """Page by page or all at once: the same codes where no page is rescaled."""
    g = torch.Generator().manual_seed(6)
    k, v = ((torch.randn(192, 2, 32, generator=g)).to(BF).cuda() for _ in range(2))
    table = torch.tensor([[1, 2, 0]], dtype=torch.int32, device="cuda")
    rope = bq.rope_table(200, 32)
    one, two = bq.KVCache.allocate(3, 2, 32), bq.KVCache.allocate(3, 2, 32)
    bq.cache_append(one, k, v, table, torch.tensor([192], dtype=torch.int32, device="cuda"), rope=rope, cu_seqlens=starts([192]))
    for i in range(0, 192, 64):
        bq.cache_append(two, k[i:i + 64], v[i:i + 64], table, torch.tensor([i + 64], dtype=torch.int32, device="cuda"), rope=rope,
                        cu_seqlens=starts([64]))
    for a, b in ((one.k, two.k), (one.v, two.v), (one.exponents, two.exponents)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    keys, values = one.read(table[0], 192)
    assert (values - v.float()).abs().max() <= 2.0 ** -4 * v.float().abs().max()
    want, _ = turned(k, torch.arange(192), rope, False)
    assert (keys.double().cpu() - want).abs().max() <= 2.0 ** -4 * want.abs().max()


def test_borders_of_the_exponents():
    table = torch.tensor([[0]], dtype=torch.int32, device="cuda")
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    for top, dtype in ((448.0, BF), (449.0, HF), (450.0, BF), (896.0, HF), (2.0 ** -33, BF), (2.0 ** -32 * 1.75, BF), (2.0 ** -60, BF),
                       (448 * 2.0 ** 40, BF), (1e30, BF), (0.0, HF), (1.75, BF), (1.7578125, HF)):
        cache = bq.KVCache.allocate(1, 1, 16)
        k = torch.zeros(1, 1, 16, dtype=dtype, device="cuda")
        k[0, 0, 3], k[0, 0, 4], k[0, 0, 5] = top, -top / 3, -0.0
        before = Snapshot(cache)
        bq.cache_append(cache, k, k, table, one)
        check_append(before, cache, k, k, table, one, [1])


def test_values_that_are_not_finite():
    g = torch.Generator().manual_seed(8)
    cache = random_cache(3, 2, 32, g)
    k, v = (torch.randn(3, 2, 32, generator=g).to(HF).cuda() for _ in range(2))
    k[0, 1, 4], v[1, 0, 3], v[2, 1] = math.nan, math.inf, -math.inf
    lengths = torch.tensor([70], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    before = Snapshot(cache)
    bq.cache_append(cache, k, v, table, lengths, cu_seqlens=starts([3]))
    check_append(before, cache, k, v, table, lengths, [3])


def test_what_the_table_does_not_hold():
    """Entries that name no page, positions past the table or before 0, tokens of no sequence."""
    g = torch.Generator().manual_seed(9)
    cache = random_cache(6, 2, 64, g)
    k, v, q = (torch.randn(420, h, 64, generator=g).to(BF).cuda() for h in (2, 2, 4))
    table = torch.tensor([[0, -1, 3], [6, 2, 1000000], [4, -2 ** 31, 2 ** 31 - 1], [5, 1, -1]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([150, 180, 260, 3], dtype=torch.int32, device="cuda")     # past the table; fewer than its tokens
    new = [140, 100, 150, 10]
    cu = starts(new) + 7                                                              # 7 tokens before, 13 after
    before = Snapshot(cache)
    rope = bq.rope_table(100, 64)                                                     # shorter than the positions
    out = bq.cache_append(cache, k, v, table, lengths, q=q, rope=rope, cu_seqlens=cu)
    torch.cuda.synchronize()
    check_append(before, cache, k, v, table, lengths, new, rope, first=7)
    positions = torch.cat([torch.arange(n - m, n) for n, m in zip(lengths.tolist(), new)])
    want, bound = turned(q[7:407], positions, rope, False)
    assert_within(out[7:407], want, bound + U16[BF] * (want.abs() + bound) + TINY[BF], "q")
    assert torch.equal(out[:7], q[:7]) and torch.equal(out[407:], q[407:])
    # starts that fall or lie outside, lengths that are no lengths: no access leaves the tensors
    whole = torch.full((8, 6 * 2 * PAGE * 64), 0x55, dtype=torch.uint8, device="cuda")
    fenced = bq.KVCache(whole[3].view(bq.KVCache.allocate(1, 1, 16).k.dtype).view(6, 2, PAGE, 64),
                        whole[5].view(cache.k.dtype).view(6, 2, 4, 64, 16), cache.exponents)
    for cu in ([0, 500, -3, 420, 420], [-5, 10, 5, 2 ** 31 - 1, 0], [0, 420, 0, 420, 0]):
        for lens in ([-1, 2 ** 31 - 1, -2 ** 31, 5], [2 ** 31 - 1] * 4, [0, 0, 0, 0], [192, 192, 192, 192]):
            bq.cache_append(fenced, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), q=q, rope=rope,
                            cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert (whole[[0, 1, 2, 4, 6, 7]] == 0x55).all()


def test_far_pages():
    # codes past 2^31 bytes
    pages = 2 ** 31 // (2 * PAGE * 128) + 5
    cache = bq.KVCache.allocate(pages, 2, 128)
    k, v = (torch.randn(70, 2, 128, device="cuda").to(BF) for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([70], dtype=torch.int32, device="cuda")
    bq.cache_append(cache, k, v, table, lengths, cu_seqlens=starts([70]))
    keys, values = cache.read(table[0], 70)
    assert (keys - k.float()).abs().max() <= 2.0 ** -4 * k.float().abs().max() and (values - v.float()).abs().max() <= 2.0 ** -4 * v.float().abs().max()


def test_stream_and_graph():
    g = torch.Generator().manual_seed(11)
    cache = random_cache(4, 2, 64, g)
    k, v, q = (torch.randn(2, h, 64, generator=g).to(BF).cuda() for h in (2, 2, 4))
    table = torch.tensor([[0, 1], [3, 2]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([60, 3], dtype=torch.int32, device="cuda")
    rope = bq.rope_table(128, 64)
    bq.cache_append(cache, k, v, table, lengths, q=q, rope=rope)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = bq.cache_append(cache, k, v, table, lengths, q=q, rope=rope)
    for i in range(8):     # replays with changed inputs, over a page's border
        lengths += 1
        k.mul_(1.3)
        before = Snapshot(cache)
        graph.replay()
        torch.cuda.synchronize()
        check_append(before, cache, k, v, table, lengths, [1, 1], rope)
        want, bound = turned(q, lengths.cpu() - 1, rope, False)
        assert_within(static, want, bound + U16[BF] * (want.abs() + bound) + TINY[BF], "q")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    before = Snapshot(cache)
    with torch.cuda.stream(s):
        bq.cache_append(cache, k, v, table, lengths, rope=rope)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    check_append(before, cache, k, v, table, lengths, [1, 1], rope)


def test_empty():
    cache = bq.KVCache.allocate(2, 2, 32)
    k = torch.zeros(0, 2, 32, dtype=BF, device="cuda")
    n = torch.tensor([5], dtype=torch.int32, device="cuda")
    q = bq.cache_append(cache, k, k, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), n, q=k, cu_seqlens=starts([0]))
    assert q.shape == (0, 2, 32)


def test_refuses():
    cache = bq.KVCache.allocate(2, 2, 32)
    k, table, n = torch.zeros(1, 2, 32, dtype=BF, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), \
        torch.ones(1, dtype=torch.int32, device="cuda")
    rope = bq.rope_table(8, 32)
    ok = dict(cache=cache, k=k, v=k, block_table=table, lengths=n)
    other = bq.KVCache.allocate(2, 1, 32)
    for kw in (dict(k=k.float()), dict(v=k.half()), dict(k=k.cpu()), dict(block_table=table.long()), dict(lengths=n.long()), dict(lengths=n.cpu()),
               dict(rope=rope.double()), dict(rope=rope[0]), dict(q=k.half()), dict(cu_seqlens=n.long()), dict(lengths=None), dict(k=k[0]),
               dict(cache=bq.KVCache(cache.k.view(torch.uint8), cache.v, cache.exponents)), dict(cache=bq.KVCache(cache.k, cache.v, None))):
        with pytest.raises(TypeError):
            bq.cache_append(**{**ok, **kw})
    for kw in (dict(cache=other), dict(k=k[:, :1]), dict(lengths=torch.ones(2, dtype=torch.int32, device="cuda")), dict(q_out=k),
               dict(cu_seqlens=starts([1, 0])), dict(q=k[:, :, :16]), dict(q=k, q_out=k[:, :1]), dict(q=k[0], rope=rope),
               dict(cache=bq.KVCache(cache.k, cache.v[:1], cache.exponents)), dict(cache=bq.KVCache(cache.k, cache.v.transpose(0, 1), cache.exponents)),
               dict(block_table=torch.zeros(2, 2, dtype=torch.int32, device="cuda")[:, :1])):
        with pytest.raises(ValueError):
            bq.cache_append(**{**ok, **kw})
    for kw in (dict(rope=bq.rope_table(8, 24)), dict(rope=bq.rope_table(8, 48)), dict(rope=rope[:0]), dict(q=torch.zeros(1, 3, 32, dtype=BF, device="cuda"))):
        with pytest.raises(bq.SvdqError):
            bq.cache_append(**{**ok, **kw})
