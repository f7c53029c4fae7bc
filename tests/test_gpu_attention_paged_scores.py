"""Scores of any size that fp32 holds, in the attention over the paged cache:
one key outweighs all others by more than every rounding, so that each query's
result is that key's value and its log-sum the key's score."""

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import TINY, U16, U32, assert_within
from tests._reference_cache import F8, PAGE, by_place, random_cache, starts, tables
from tests.test_gpu_attention_paged import plan

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

# (new tokens, lengths, heads_q, heads_k, head_dim, rows of a tile, shares)
CASES = [([1, 1], [200, 1], 8, 2, 128, 16, 0), ([5], [300], 8, 2, 64, 32, 0), ([1, 1], [3000, 70], 8, 2, 128, 16, 512),
         ([40], [3000], 8, 2, 128, 32, 512), ([700, 300], [1290, 365], 32, 8, 128, 256, 0), ([1000], [1000], 32, 8, 64, 128, 0)]


def check(case, dtype, sign, power, far):
    """Every key scores 2 s but one, which scores s (sign < 0), or s / 2 beside
    s; |s| near 2^power.  `far`: the one lies in the middle, for queries that
    see all keys, else it is the first."""
    new, lens, hq, hk, d, rows, shares = case
    print("attention_paged", case, dtype, sign, power, far, flush=True)
    g = torch.Generator().manual_seed(sum(new) + d)
    table, pages = tables(lens, g)
    assert plan(sum(new), len(new), table.shape[1], hq, hk, d) == (rows, shares)
    cache = random_cache(pages, hk, d, g)
    # |s| = d 43200 224 scale 2^e
    e = max(0, min(40, power - 30))
    cache.exponents[:, :, 0] = e
    scale = 1.37 * 2.0 ** power / (d * 43200 * 224 * 2.0 ** e)
    codes = torch.tensor([-448.0, -224.0] if sign < 0 else [224.0, 448.0]).to(F8).view(torch.uint8)
    cache.k.view(torch.uint8)[:] = int(codes[0])
    one = [n // 2 if far else 0 for n in lens]
    place = torch.tensor([i % PAGE for i in one])
    page = table.cpu()[torch.arange(len(lens)), torch.tensor([i // PAGE for i in one])].long()
    cache.k.view(torch.uint8)[page.cuda(), :, place.cuda()] = int(codes[1])
    q = torch.full((sum(new), hq, d), 43200.0, dtype=dtype, device="cuda")
    o, lse = bq.attention_paged(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_seqlens_q=starts(new),
                                causal=not far, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    value = by_place(cache.v).cpu()[page, :, place].view(F8).double() * torch.exp2(cache.exponents.cpu()[page, :, 1].double())[:, :, None]
    value = value.repeat_interleave(hq // hk, 1).repeat_interleave(torch.tensor(new), 0)
    s = d * float(q[0, 0, 0]) * float(codes[1:].view(F8)) * 2.0 ** e * scale
    # the weight and the result are rounded to 16 bits once each; its product
    # with the value, the sum and the quotient in fp32
    assert_within(o, value, (2 * U16[dtype] + U16[dtype] ** 2 + 16 * U32) * value.abs() + TINY[dtype], "o")
    # d products and as many sums, the scale, the exponent, the logarithm
    assert_within(lse, torch.full(lse.shape, s, dtype=torch.float64), torch.full(lse.shape, (d + 16) * U32 * abs(s)), "lse")


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("far", [False, True])
def test_one_key_outweighs_all(case, dtype, far):
    for power in (14, 18, 20, 22, 24, 28, 33, 60, 90):
        check(case, dtype, -1, power, far)
        check(case, dtype, 1, power, far)
    check(case, dtype, 1, 120, far)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("far", [False, True])
def test_scores_far_below_zero(case, dtype, far):
    for power in (98, 99, 100, 110, 120, 125):      # 2 s log2 e from -2^99.6 to -2^127
        check(case, dtype, -1, power, far)
