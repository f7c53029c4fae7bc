"""RMS norm of rows whose squares leave fp32's range: finite rows of any size,
with an eps that matters to them or not."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import TINY, U16, assert_within
from tests._reference8 import blocks, code_bound
from tests.test_gpu_rms_norm import check

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

# every layout of a row: 16 lanes, a wave, four and sixteen
WIDTHS = (16, 77, 128, 512, 1000, 1024, 2048, 4096, 8192, 16384, 40000, 65536)


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("power", [52, 57, 60, 64, 80, 120])
def test_large_rows(k, power):
    check(3, k, BF, std=2.0 ** power)
    check(3, k, BF, residual=True, std=2.0 ** power, weight=False)


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("power", [-35, -60, -66, -72, -80, -100, -110])
def test_small_rows(k, power):
    for eps in (0.0, 2.0 ** (2 * power), 1e-20, 1e-6):
        eps = float(torch.tensor(eps, dtype=torch.float32))      # as the norm receives it: from 2^-150 on zero
        check(3, k, BF, residual=eps == 0.0, std=2.0 ** power, eps=eps)


def test_more_rows_than_cus():
    for k in (1536, 4096):
        check(300, k, BF, std=2.0 ** 100)
        check(300, k, BF, std=2.0 ** -80, eps=0.0)


def test_rows_of_every_size_together():
    """Rows that need another scale stand beside rows that do not, and rows of zeros."""
    g = torch.Generator().manual_seed(1)
    for k in (64, 128, 496, 4096):
        size = torch.exp2(torch.randint(-100, 120, (64, 1), generator=g).double())
        x = (torch.randn(64, k, generator=g).double() * size).to(BF).cuda()
        x[5] = 0.0
        check(64, k, BF, x=x, eps=1e-30)
    # a value far above the others of its row
    for k in (64, 4096):
        x = torch.randn(4, k, generator=g).to(BF).cuda()
        x[:, 7] = torch.tensor([1e38, -3e38, 1e30, 1e20])
        check(4, k, BF, x=x)


def test_ends_of_the_range():
    for k in (16, 77, 1024, 4096, 65536):
        for value in (3.3e38, -3e38, 2.0 ** 127, 2.0 ** -126, -2.0 ** -126, 2.0 ** -130, 2.0 ** -133):
            check(3, k, BF, x=torch.full((3, k), value, dtype=BF, device="cuda"), eps=0.0)
            check(3, k, BF, x=torch.full((3, k), value, dtype=BF, device="cuda"), eps=1e38)


def test_not_finite():
    x = torch.randn(6, 512, device="cuda").to(BF) * 2.0 ** 70
    clean = bq.rms_norm(x)
    x[2, 5], x[4, 9] = math.nan, math.inf
    y = bq.rms_norm(x)
    assert torch.equal(y[[0, 1, 3, 5]], clean[[0, 1, 3, 5]]) and y[2].isnan().all() and y[4, 9].isnan()
    assert (y[4, :9] == 0).all() and (y[4, 10:] == 0).all()
    zero = torch.zeros(2, 512, dtype=BF, device="cuda")
    assert bq.rms_norm(zero, eps=0.0).isnan().all() and (bq.rms_norm(zero, eps=1e-30) == 0).all()      # 0 / 0; 0


def test_fp16_rows():
    for k in (128, 4096, 65536):
        check(3, k, HF, x=torch.full((3, k), 65504.0, dtype=HF, device="cuda"), residual=False)
        check(3, k, HF, x=torch.full((3, k), 2.0 ** -24, dtype=HF, device="cuda"), eps=0.0)
