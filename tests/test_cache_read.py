"""KVCache.read shows what the attention sees (CPU)."""

import pytest
import torch

import bit_quantized_diffusion_amd as bq


def cache(pages=4, heads=2, d=16):
    g = torch.Generator().manual_seed(3)
    c = bq.KVCache.allocate(pages, heads, d, device="cpu")
    for t in (c.k, c.v):
        t.copy_((torch.randn(t.shape, generator=g) * 50).to(t.dtype))
    c.exponents.copy_(torch.randint(-9, 3, c.exponents.shape, generator=g).to(torch.int8))
    return c


def plain(c, page, place, head):
    """(key, value) of a place, by the layout."""
    ek, ev = (2.0 ** max(-40, min(40, int(e))) for e in c.exponents[page, head])
    k = c.k.view(torch.uint8)[page, head, place].view(c.k.dtype).float()
    v = c.v.view(torch.uint8)[page, head, place // 4 % 4, :, place // 16 * 4 + place % 4].contiguous().view(c.v.dtype).float()
    return k * ek, v * ev


def same(c, row, length):
    keys, values = c.read(torch.tensor(row, dtype=torch.int32), length)
    _, heads, _, d = c.k.shape
    assert keys.shape == values.shape == (length, heads, d) and keys.dtype == values.dtype == torch.float32
    for j in range(length):
        page = row[j // bq.PAGE] if j // bq.PAGE < len(row) else -1
        for h in range(heads):
            k, v = plain(c, page, j % bq.PAGE, h) if 0 <= page < c.k.shape[0] else (torch.zeros(d), torch.zeros(d))
            assert torch.equal(keys[j, h], k) and torch.equal(values[j, h], v), (j, h)


@pytest.mark.parametrize("length", [1, 63, 64, 65, 150, 192])
def test_layout(length):
    same(cache(), [2, 0, 3], length)


def test_exponents_past_their_range():
    c = cache()
    c.exponents[2], c.exponents[0] = 100, -128
    same(c, [2, 0, 3], 150)


def test_pages_that_are_not_there():
    c = cache()
    c.k.view(torch.uint8)[3], c.v.view(torch.uint8)[3] = 0x7F, 0x7F       # the last page holds NaN
    same(c, [2, -1, 0], 150)
    same(c, [-1, 4, 2 ** 31 - 1, 1, -2 ** 31], 310)


def test_lengths():
    same(cache(), [2, 0, 3], 0)
    same(cache(), [2], 100)          # past the table
    same(cache(), [], 0)


def test_length_from_a_tensor():
    c, row = cache(), torch.tensor([2, 0, 3], dtype=torch.int32)
    for length in (torch.tensor([70], dtype=torch.int32)[0], torch.tensor(70)):
        for a, b in zip(c.read(row, length), c.read(row, 70)):
            assert torch.equal(a, b)
