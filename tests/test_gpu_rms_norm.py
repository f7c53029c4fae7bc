"""GPU parity of the root-mean-square norm, its 8-bit output and the activation
quantizer against plain 64-bit references."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import TINY, U16, assert_within
from tests._reference8 import F8, blocks, code_bound, quantize_plain, rms_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def matrix(gen, m, k, dtype, pad=0, std=1.0):
    return (torch.randn(m, k + pad, generator=gen) * std).to(dtype).cuda()[:, :k]


def check(m, k, dtype, residual=False, weight=True, pad=0, std=1.0, eps=1e-6, x=None, fp8=None):
    print("rms_norm", m, k, dtype, residual, weight, pad, std, flush=True)
    g = torch.Generator().manual_seed(m + k)
    x = matrix(g, m, k, dtype, pad, std) if x is None else x
    r = matrix(g, m, k, dtype, pad, 2 * std) if residual else None
    w = (torch.randn(k, generator=g) * 0.2 + 1).to(dtype).cuda() if weight else None
    h, bound_h, y, bound_y = rms_reference(x, r, w, eps)
    got = bq.rms_norm(x, w, residual=r, eps=eps)
    got_y, got_h = got if residual else (got, None)
    assert_within(got_y, y, bound_y + U16[dtype] * (y.abs() + bound_y) + TINY[dtype], f"{m}x{k}")
    if residual:
        assert_within(got_h, h, bound_h, f"sum {m}x{k}")
    if k % 16:
        return
    got = bq.rms_norm_fp8(x, w, residual=r, eps=eps)
    codes, scales = got[:2]
    assert codes.shape == (m, k) and codes.dtype == F8 and scales.shape == (blocks(k), m)
    if residual:
        assert torch.equal(got[2], got_h)
    rel = (bound_y / y.abs().clamp(min=1e-300)).amax()
    pad_y = torch.nn.functional.pad(y, (0, blocks(k) * 128 - k)).view(m, -1, 128)
    s = pad_y.abs().amax(2).clamp(min=2.0 ** -100) / 448
    assert_within(scales.t(), s, s * (rel + 4 * 2.0 ** -24), f"scales {m}x{k}")
    want = (pad_y / s[:, :, None]).view(m, -1)[:, :k]
    assert_within(codes.float(), want, code_bound(want, want.abs() * (2 * rel + 8 * 2.0 ** -24)), f"codes {m}x{k}")


# around every switch of the row's layout, odd sizes and short last blocks among them
@pytest.mark.parametrize("k", [1, 7, 8, 9, 16, 48, 127, 128, 129, 144, 255, 256, 512, 520, 1024, 1040, 2048, 2064, 4095, 4096, 4112, 8192,
                               8208, 12288, 16384, 16400, 40000, 65535, 65536])
def test_widths(k):
    for dtype in (BF, HF):
        check(3, k, dtype, residual=True)
        check(5, k, dtype, weight=False)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 257, 1000])
def test_rows(m):
    check(m, 144, BF, residual=True)
    check(m, 4096, HF)


@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strided_and_misaligned(pad):
    for k in (64, 77, 1008, 5008):
        check(9, k, BF, residual=True, pad=pad)
        check(9, k, HF, pad=pad)


def test_extreme_rows():
    for k in (112, 4096):
        check(4, k, BF, std=1e15)
        check(4, k, BF, residual=True, std=1e-15, eps=0.0)
        check(4, k, HF, x=torch.zeros(4, k, dtype=HF, device="cuda"))          # eps alone
        check(4, k, BF, x=torch.full((4, k), 3.0, dtype=BF, device="cuda"))
    x = torch.randn(6, 512, device="cuda").to(BF)
    clean, codes = bq.rms_norm(x), bq.rms_norm_fp8(x)
    x[2, 5], x[4, 9] = math.nan, math.inf
    keep = [0, 1, 3, 5]
    y, (yq, ys) = bq.rms_norm(x), bq.rms_norm_fp8(x)
    assert torch.equal(y[keep], clean[keep]) and y[2].isnan().all() and y[4, 9].isnan()
    assert torch.equal(yq[keep].view(torch.uint8), codes[0][keep].view(torch.uint8)) and torch.equal(ys[:, keep], codes[1][:, keep])
    assert yq.float()[2].isnan().all() and yq.float()[4, 9].isnan()


def test_in_place():
    g = torch.Generator().manual_seed(3)
    for k in (77, 520, 9000):
        x, r, w = matrix(g, 9, k, BF), matrix(g, 9, k, BF), matrix(g, 1, k, BF)[0]
        y, h = bq.rms_norm(x, w, residual=r)
        r1 = r.clone()
        y1, h1 = bq.rms_norm(x, w, residual=r1, residual_out=r1)
        assert h1 is r1 and torch.equal(r1, h) and torch.equal(y1, y)
        x1, r1 = x.clone(), r.clone()
        y1, h1 = bq.rms_norm(x1, w, residual=r1, out=x1, residual_out=r1)
        assert y1 is x1 and torch.equal(x1, y) and torch.equal(r1, h)
    assert bq.rms_norm(x[:0], w).shape == (0, 9000)
    q, s = bq.rms_norm_fp8(matrix(g, 4, 160, BF)[:0])
    assert q.shape == (0, 160) and s.shape == (2, 0)


@pytest.mark.parametrize("m,k", [(1, 16), (1, 128), (7, 144), (33, 4096), (1000, 1552), (3, 70000 // 16 * 16)])
def test_quantize(m, k):
    g = torch.Generator().manual_seed(k)
    for dtype, pad in ((BF, 0), (HF, 5)):
        x = matrix(g, m, k, dtype, pad, 3.0)
        x[0, : k // 2] = 0
        x[m // 2, 3] = 500.0
        q, s = bq.quantize_fp8(x)
        want_q, want_s = quantize_plain(x)
        assert torch.equal(s.cpu(), want_s)
        assert torch.equal(q.cpu().view(torch.uint8), want_q.view(torch.uint8))


def test_quantize_extremes():
    x = torch.randn(5, 256, device="cuda").to(BF)
    x[0], x[1], x[2, 7], x[3, 200] = 0.0, x[1] * 2.0 ** -120, math.nan, math.inf
    x[4] *= 1e30
    q, s = bq.quantize_fp8(x)
    want_q, want_s = quantize_plain(x)
    assert torch.equal(s.cpu(), want_s)
    q, want = q.cpu().float(), want_q.float()
    assert torch.equal(q.isnan(), want.isnan()) and torch.equal(q.nan_to_num(0), want.nan_to_num(0))
    assert q[2, 7].isnan() and q[3, 200].isnan() and s[1, 3].isinf()


def test_stream_and_graph():
    x, r = torch.randn(64, 2048, device="cuda").to(BF), torch.randn(64, 2048, device="cuda").to(BF)
    want = bq.rms_norm_fp8(x, residual=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = bq.rms_norm_fp8(x, residual=r)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = bq.rms_norm_fp8(x, residual=r)
        codes = bq.quantize_fp8(x)
    keep = x.clone()
    for i in range(3):
        x.copy_(keep * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*static, *codes), (*bq.rms_norm_fp8(x, residual=r), *bq.quantize_fp8(x))):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_far_rows():
    ld, m = 2 ** 25, 70
    buf = torch.empty(ld * m, dtype=BF, device="cuda")
    x = buf.as_strided((m, 208), (ld, 1))
    x.copy_(torch.randn(m, 208))
    check(m, 208, BF, x=x)
    q, s = bq.quantize_fp8(x)
    want_q, want_s = quantize_plain(x)
    assert torch.equal(q.cpu().view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s.cpu(), want_s)


def test_refuses():
    x = torch.zeros(4, 64, device="cuda", dtype=BF)
    for call in (lambda: bq.rms_norm(x.float()), lambda: bq.rms_norm(x, torch.ones(64, device="cuda")), lambda: bq.quantize_fp8(x.float()),
                 lambda: bq.rms_norm(x, residual=x.half()), lambda: bq.rms_norm_fp8(None), lambda: bq.rms_norm(x, out=3)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: bq.rms_norm(x, torch.ones(63, device="cuda", dtype=BF)), lambda: bq.rms_norm(x, residual=x[:3]),
                 lambda: bq.rms_norm(x, residual_out=x), lambda: bq.rms_norm_fp8(x[:, :40]), lambda: bq.rms_norm(x, out=x[:2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bq.rms_norm(x, eps=-1.0), lambda: bq.rms_norm(x, eps=math.nan), lambda: bq.quantize_fp8(x[:, :40]),
                 lambda: bq.rms_norm(torch.zeros(1, 65537, device="cuda", dtype=BF))):
        with pytest.raises(bq.SvdqError):
            call()
