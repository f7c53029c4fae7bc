"""GPU tests of attention's rows without keys: queries that causal masking
leaves none, whatever the values beside them hold."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def cu(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d", [
    ([40], [20], 2, 1, 128),               # tiles of 32 rows, one workgroup through all keys
    ([40, 1], [20, 3000], 2, 2, 64),       # the same with equal shares of the keys over workgroups
    ([300], [200], 3, 3, 64),              # tiles of 128 rows
    ([300, 130], [200, 90], 2, 1, 72),
    ([1000], [800], 2, 2, 128),            # the keys in two parts within a workgroup
    ([1500], [1200], 2, 1, 40),            # and split over workgroups
])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_rows_without_keys_are_zero_beside_values_that_are_not_finite(lens_q, lens_k, hq, hk, d, dtype):
    """Causal with more queries than keys: the first len_q - len_k rows see no
    key, and share tiles with rows that see a NaN and an infinity."""
    g = torch.Generator().manual_seed(3)
    q = torch.randn(sum(lens_q), hq, d, generator=g).to(dtype).cuda()
    k = torch.randn(sum(lens_k), hk, d, generator=g).to(dtype).cuda()
    v = torch.randn(sum(lens_k), hk, d, generator=g).to(dtype).cuda()
    v[0], v[1], v[lens_k[0] - 1] = math.nan, math.inf, -math.inf
    empty = torch.zeros(sum(lens_q), dtype=torch.bool)
    q0 = 0
    for nq, nk in zip(lens_q, lens_k):
        empty[q0:q0 + max(nq - nk, 0)] = True
        q0 += nq
    assert empty.any()
    for ws in ("auto", None):
        print("rows without keys", lens_q, lens_k, hq, hk, d, dtype, ws, flush=True)
        o, lse = bq.attention(q, k, v, cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k), causal=True, return_lse=True, workspace=ws)
        o, lse = o.cpu(), lse.cpu()
        assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all()
        assert lse[~empty].isfinite().all()
        assert o[lens_q[0] - 1].isnan().all()   # the last query sees them all
