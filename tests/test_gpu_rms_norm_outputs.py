"""The norm's two results need a place each."""

import pytest
import torch

import bit_quantized_diffusion_amd as bq

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rows(flat, first, stride, m=6):
    return flat.as_strided((m, 96), (stride, 1), first)


# first element and row stride of each result in one buffer
@pytest.mark.parametrize("a,b", [
    ((0, 256), (0, 256)), ((0, 256), (95, 256)), ((0, 256), (256, 256)), ((0, 256), (1280 + 95, 256)), ((200, 256), (406, 256)),
    ((0, 96), (0, 256)), ((1300, 96), (0, 256)), ((500, 96), (980, 1000)),
])
def test_refuses_one_place_for_both(a, b):
    x, r = (torch.randn(6, 96, device="cuda").to(BF) for _ in range(2))
    flat = torch.full((8192,), 7.0, dtype=BF, device="cuda")
    for one, two in ((a, b), (b, a)):
        with pytest.raises(ValueError):
            bq.rms_norm(x, residual=r, out=rows(flat, *one), residual_out=rows(flat, *two))
    with pytest.raises(ValueError):
        bq.rms_norm(x[:1], residual=r[:1], out=rows(flat, 0, 96, 1), residual_out=rows(flat, 95, 96, 1))
    torch.cuda.synchronize()
    assert (flat == 7).all()


@pytest.mark.parametrize("a,b", [
    ((0, 256), (96, 256)), ((160, 256), (0, 256)), ((200, 256), (40, 256)), ((0, 256), (1280 + 96, 256)), ((0, 512), (256, 512)),
    ((0, 96), (576, 96)), ((0, 96), (576, 256)), ((0, 256), (100, 512)), ((1000, 1000), (420, 96)),
])
def test_results_beside_each_other(a, b):
    x, r = (torch.randn(6, 96, device="cuda").to(BF) for _ in range(2))
    y, h = bq.rms_norm(x, residual=r)
    for one, two in ((a, b), (b, a)):
        flat = torch.full((8192,), 7.0, dtype=BF, device="cuda")
        out, total = rows(flat, *one), rows(flat, *two)
        bq.rms_norm(x, residual=r, out=out, residual_out=total)
        assert torch.equal(out, y) and torch.equal(total, h)
        flat[torch.cat([rows(torch.arange(8192, device="cuda"), *at).reshape(-1) for at in (a, b)])] = 7.0
        assert (flat == 7).all()
    # one row after the other, and a single row
    x1 = x[:1].clone()
    got = bq.rms_norm(x1, residual=r[:1], out=x1, residual_out=rows(flat, 0, 96, 1))
    assert torch.equal(got[0], y[:1]) and torch.equal(got[1], h[:1])
