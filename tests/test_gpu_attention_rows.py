"""GPU tests of attention's rows without keys: queries that causal masking
leaves none, whatever the values beside them hold, and queries outside every
sequence."""

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


# (lens_q, lens_k, heads_q, heads_k, head_dim, causal), one for each schedule
SCHEDULES = [
    ([20, 0, 31], [40, 9, 100], 4, 2, 128, True),         # tiles of 32 rows, one workgroup through all keys
    ([300, 200], [200, 90], 3, 3, 64, True),
    ([1] * 70, [0, 5, 64] * 23 + [3000], 2, 1, 40, True),   # more sequences than the lanes of a wave hold
    ([1, 2, 1], [900, 0, 3000], 4, 2, 64, False),         # the same with equal shares of the keys over workgroups
    ([600, 500], [700, 400], 3, 3, 64, True),             # tiles of 128 rows
    ([1000], [900], 2, 2, 128, False),                    # the keys in two parts within a workgroup
    ([700, 500], [2000, 2100], 2, 1, 72, False),          # and split over workgroups
    ([1100, 0, 1301], [1900, 40, 1300], 16, 8, 64, False),    # tiles of 256 rows
]
# (rows of a tile, parts, whether split, whether equal shares) of each
PLANS = [(32, 1, False, False)] * 3 + [(32, 1, False, True), (128, 1, False, False), (128, 2, False, False),
                                       (128, 2, True, False), (256, 1, False, False)]


def packed(lens_q, lens_k, hq, hk, d, dtype, front, back):
    """q, k and v with `front` and `back` tokens of padding around the sequences."""
    g = torch.Generator().manual_seed(7)
    pad = front + back
    q = torch.randn(sum(lens_q) + pad, hq, d, generator=g).to(dtype).cuda()
    k = torch.randn(sum(lens_k) + pad, hk, d, generator=g).to(dtype).cuda()
    v = torch.randn(sum(lens_k) + pad, hk, d, generator=g).to(dtype).cuda()
    return q, k, v, cu(lens_q) + front, cu(lens_k) + front


@pytest.mark.parametrize("front,back", [(0, 1), (3, 0), (0, 300), (41, 70)])
@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d,causal", SCHEDULES)
def test_queries_that_no_sequence_holds(lens_q, lens_k, hq, hk, d, causal, front, back):
    """Padding around the sequences gives zeros, and nothing of what the
    output or the workspace held before."""
    q, k, v, cu_q, cu_k = packed(lens_q, lens_k, hq, hk, d, BF, front, back)
    n = sum(lens_q)
    want, want_lse, bo, bl = attention_reference(q[front:front + n], k[front:front + sum(lens_k)], v[front:front + sum(lens_k)],
                                                 lens_q, lens_k, causal, d ** -0.5)
    size = bq.attention_workspace_size(q.shape[0], k.shape[0], len(lens_q), hq, hk, d)
    for ws in (torch.full((max(size, 16),), 0x42, dtype=torch.uint8, device="cuda"), None):
        print("padding", lens_q[:5], lens_k[:5], hq, hk, d, causal, front, back, ws is None, flush=True)
        out = torch.full_like(q, 7.0)
        stale = torch.full((q.shape[0], hq), 7.0, device="cuda")   # what a new lse may lie in
        del stale
        o, lse = bq.attention(q, k, v, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k, causal=causal, return_lse=True, workspace=ws, out=out)
        assert_within(o[front:front + n], want, bo, "o")
        assert_within(lse[front:front + n], want_lse, bl, "lse")
        for a, b in ((0, front), (front + n, front + n + back)):
            assert (o[a:b] == 0).all() and (lse[a:b] == -math.inf).all()


LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d,causal", SCHEDULES)
def test_starts_that_fall_or_lie_outside_are_cut(lens_q, lens_k, hq, hk, d, causal):
    """Whatever the starts hold, only the output is written, and the next
    call is right."""
    q, k, v, cu_q, cu_k = packed(lens_q, lens_k, hq, hk, d, BF, 0, 0)
    tq, tk, batch = q.shape[0], k.shape[0], len(lens_q)
    size = bq.attention_workspace_size(tq, tk, batch, hq, hk, d)
    ws = torch.full((size + 4096,), 0x42, dtype=torch.uint8, device="cuda")
    whole = torch.full((tq + 64, hq, d), 7.0, dtype=BF, device="cuda")

    def bad(good, total, i):
        n = batch + 1
        s = good.tolist()
        return [[HIGH] * n, [LOW] * n, s[::-1], [total, 0] * (n // 2) + [total] * (n % 2), [0] + [HIGH] * (n - 1),
                [LOW] + s[1:], s[:-1] + [LOW], s[:-1] + [total + 1]][i]

    for i in range(8):
        for j in (i, (i + 3) % 8):
            print("starts", lens_q[:5], lens_k[:5], hq, hk, d, causal, i, j, flush=True)
            starts = [torch.tensor(bad(c, t, n), dtype=torch.int32, device="cuda") for c, t, n in ((cu_q, tq, i), (cu_k, tk, j))]
            bq.attention(q, k, v, cu_seqlens_q=starts[0], cu_seqlens_k=starts[1], causal=causal, workspace=ws[:size], out=whole[32:-32])
            torch.cuda.synchronize()
            assert (whole[:32] == 7).all() and (whole[-32:] == 7).all() and (ws[size:] == 0x42).all()
    o = bq.attention(q, k, v, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k, causal=causal, workspace=ws, out=whole[32:-32])
    want, _, bo, _ = attention_reference(q, k, v, lens_q, lens_k, causal, d ** -0.5)
    assert_within(o, want, bo, "o")
