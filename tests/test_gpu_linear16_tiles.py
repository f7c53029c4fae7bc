"""GPU parity of the 16-bit linear's tile shapes against a plain 64-bit
reference: each with remainders of rows, channels and K, in one piece and
split, its plan pinned."""

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._plans import linear16_plan
from tests._reference16 import assert_within, linear16_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


# (m, n, k, aligned): rows of a tile, channels, waves, splits
TILES = {
    (4097, 3000, 2056, True): (256, 256, 8, 1),
    (4500, 3081, 3080, True): (256, 256, 8, 1),
    (1000, 4101, 200, True): (128, 128, 4, 1),
    (2500, 2051, 4104, True): (128, 128, 4, 1),
    (4097, 520, 520, True): (128, 128, 8, 1),
    (2500, 4101, 1032, True): (128, 128, 8, 1),
    (333, 520, 136, True): (64, 64, 4, 1),
    (500, 4100, 8200, True): (128, 128, 4, 2),
    (200, 3001, 8200, True): (128, 128, 8, 5),
    (257, 779, 3080, True): (64, 64, 4, 4),
    (1500, 3000, 1023, False): (128, 128, 4, 1),
    (2900, 4333, 65, False): (128, 128, 4, 1),
    (333, 3080, 8191, False): (128, 128, 4, 4),
    (200, 2051, 8191, False): (128, 128, 4, 8),
    (333, 779, 2049, False): (64, 64, 4, 3),
    (33, 17, 9, False): (64, 64, 4, 1),
}


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("m,n,k,aligned", list(TILES))
def test_tile_shapes(m, n, k, aligned, dtype):
    assert linear16_plan(m, n, k, aligned) == TILES[m, n, k, aligned]
    g = torch.Generator().manual_seed(m + n + k)

    def mat(r, c, pad=0, std=1.0):
        return (torch.randn(r, c + pad, generator=g) * std).to(dtype).cuda()[:, :c]

    x, w, b = mat(m, k, 8 if aligned else 1), mat(n, k, std=k ** -0.5), mat(1, n, std=0.5)[0]
    # a gate whose groups end inside tiles, and one for all rows; results in rows that allow wide stores, and in others
    rows = m // 3 + 1
    gates, res = mat(3, n, 3), mat(m, n)
    for act, gate, group_rows, residual, pad in (("gelu", gates, rows, res, 0), ("none", gates[0], None, None, -n % 8),
                                                 ("silu", None, None, mat(m, n, 8 - n % 8), 5)):
        print("linear16", m, n, k, dtype, act, pad, flush=True)
        whole = torch.full((m, n + pad), 5.0, dtype=dtype, device="cuda")
        y = bq.linear16(x, w, b, activation=act, gate=gate, residual=residual, group_rows=group_rows, out=whole[:, :n])
        torch.cuda.synchronize()
        assert (whole[:, n:] == 5).all()
        want, bound = linear16_reference(x, w, b, act, gate, residual, group_rows)
        assert_within(y, want, bound, f"{m}x{n}x{k} {act}")


@pytest.mark.parametrize("m,n,k,aligned", [c for c in TILES if TILES[c][0] >= 128])
def test_nan_stays_in_its_row_and_channel(m, n, k, aligned):
    x, w = torch.randn(m, k, device="cuda").to(BF), (torch.randn(n, k, device="cuda") * k ** -0.5).to(BF)
    clean = bq.linear16(x, w)
    x[m - 1, k - 1], w[n - 1, 0] = float("nan"), float("inf")
    y = bq.linear16(x, w)
    assert torch.equal(y[:-1, :-1], clean[:-1, :-1])
    assert y[-1].isnan().all() and not y[:-1, -1].isfinite().any()
