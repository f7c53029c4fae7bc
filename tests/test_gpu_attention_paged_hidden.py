"""Queries that see no key get zeros from the attention over the paged cache,
also where values within their sequence's length are NaN (as the append makes
them of what is not finite)."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference_cache import random_cache, starts, tables
from tests.test_gpu_attention_paged import plan

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

# (new tokens, lengths, heads_q, heads_k, head_dim, schedule), with more tokens
# than keys.  In the third, tiles of three pages count 7 on the line and a share
# is 8: the first rows' tiles of heads 5 and 6 are cut behind their first and
# second page, and joined.
CASES = [
    ([5], [3], 4, 2, 64, (16, 0)), ([20, 3], [3, 2], 4, 2, 128, (32, 0)),
    ([140, 1, 1, 1, 1], [130, 1300, 1300, 1300, 1300], 8, 8, 128, (32, 512)), ([3, 2], [2, 1200], 4, 2, 64, (16, 512)),
    # few rows among many, and one key for many rows
    ([700, 8, 300], [690, 5, 1], 32, 8, 128, (256, 0)), ([900, 8, 300], [890, 5, 1], 32, 8, 64, (128, 0)),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_hidden_rows_beside_nan(case, dtype):
    new, lens, hq, hk, d, schedule = case
    print("attention_paged", case, dtype, flush=True)
    g = torch.Generator().manual_seed(sum(new) + d)
    table, pages = tables(lens, g)
    assert plan(sum(new), len(new), table.shape[1], hq, hk, d) == schedule
    cache = random_cache(pages, hk, d, g)
    q = torch.randn(sum(new), hq, d, generator=g).to(dtype).cuda()
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def call():
        return bq.attention_paged(q, cache, table, lengths, cu_seqlens_q=starts(new), scale=2.0 ** -12, return_lse=True)

    _, want_lse = call()
    cache.v.view(torch.uint8)[table[:, 0].long(), :, 0, :, 0] = 0x7F      # the first key of every sequence
    o, lse = call()
    torch.cuda.synchronize()
    hidden = torch.cat([torch.arange(n) < n - length for n, length in zip(new, lens)])
    assert hidden.any() and not hidden.all()
    assert (o[hidden] == 0).all() and (lse[hidden] == -math.inf).all()
    assert o[~hidden].isnan().all() and lse[~hidden].isfinite().all() and torch.equal(lse, want_lse)
