"""GPU parity of the block-scaled 8-bit linear against a plain 64-bit
reference on the same codes."""

import ctypes
import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import assert_within
from tests._reference8 import F8, blocks, gemm_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def operands(m, n, k, seed=0):
    """Codes over the whole range of e4m3 and scales that differ from block to block."""
    g = torch.Generator().manual_seed(m * 7 + n * 3 + k + seed)

    def codes(r):
        return (torch.randn(r, k, generator=g) * 90).clamp(-448, 448).to(F8).cuda()

    xs = (torch.rand(blocks(k), m, generator=g) + 0.5) * 2.0 ** -6
    ws = (torch.rand(blocks(n), blocks(k), generator=g) + 0.5) * 2.0 ** -9
    return codes(m), xs.cuda(), codes(n), ws.cuda(), g


def check(m, n, k, dtype=BF, act="none", bias=False, gate=0, residual=False, pad=0):
    print("gemm_fp8", m, n, k, dtype, act, bias, gate, residual, pad, flush=True)
    xq, xs, wq, ws, g = operands(m, n, k)

    def mat(r, c, s=1.0):
        return (torch.randn(r, c + pad, generator=g) * s).to(dtype).cuda()[:, :c]

    b = mat(1, n)[0] if bias else None
    ga = mat(gate, n, 0.5) if gate else None
    r = mat(m, n) if residual else None
    out = None
    if pad:
        whole = torch.full((m, n + pad), 5.0, dtype=dtype, device="cuda")
        out = whole[:, :n]
    rows = -(-m // gate) if gate else None
    y = bq.gemm_fp8(xq, xs, wq, ws, b, dtype=dtype, activation=act, gate=ga, residual=r, group_rows=rows, out=out)
    torch.cuda.synchronize()
    assert y.shape == (m, n) and y.dtype == dtype
    if pad:
        assert (whole[:, n:] == 5).all()
    want, bound, expected = gemm_reference(xq, xs, wq, ws, b, act, ga, r, rows, dtype)
    assert_within(y, want, bound, f"{m}x{n}x{k}")
    if m * n >= 4096:   # enough results for their root mean square to be near the expected one
        off = float((y.cpu().double() - want).norm())
        assert off <= 1.2 * expected, (off, expected)
    return y


@pytest.mark.parametrize("m", [1, 2, 8, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("n,k", [(1, 16), (15, 128), (130, 144), (257, 1040), (512, 4096), (64, 12288)])
def test_few_rows(m, n, k):
    check(m, n, k, BF if m % 2 else HF, bias=m % 3 == 0, residual=m % 4 == 0)


@pytest.mark.parametrize("m", [33, 63, 64, 65, 127, 129, 300, 513])
@pytest.mark.parametrize("n,k", [(1, 128), (63, 16), (64, 256), (129, 400), (256, 2048), (520, 384)])
def test_tiles(m, n, k):
    check(m, n, k, HF if m % 2 else BF, residual=m % 3 == 0)


def plan(m, n, k):
    out = (ctypes.c_int32 * 3)()
    bq.check(bq.lib.svdq_debug_gemm_fp8_plan(m, n, k, out))
    return tuple(out)


# every tile shape (rows, channels, waves), with remainders on every side
SHAPES = {(13, 100, 144): (16, 16, 8), (9, 13630, 400): (16, 32, 2), (22, 117, 272): (32, 16, 8), (17, 4259, 144): (32, 32, 8),
          (75, 117, 1168): (64, 16, 8), (67, 2053, 224): (64, 32, 8), (65, 4108, 208): (64, 64, 8), (641, 5412, 224): (128, 128, 4),
          (322, 5466, 192): (128, 128, 8), (1281, 5901, 208): (160, 256, 8), (4484, 2063, 176): (192, 256, 8),
          (3655, 3090, 160): (224, 256, 8), (4267, 3093, 1040): (256, 256, 8), (4275, 3075, 224): (288, 256, 8)}


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_every_tile_shape(m, n, k):
    assert plan(m, n, k) == SHAPES[m, n, k]
    check(m, n, k)
    check(m, n, k, HF, act="gelu", bias=True, gate=1, residual=True)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_epilogue(act):
    for m, n, k in ((5, 96, 256), (100, 200, 256), (600, 1024, 384)):
        for dtype in (BF, HF):
            check(m, n, k, dtype, act=act, bias=True)
            check(m, n, k, dtype, act=act, gate=1, residual=True)
            check(m, n, k, dtype, act=act, bias=True, gate=3, residual=True)
            check(m, n, k, dtype, act=act, gate=m)


@pytest.mark.parametrize("pad", [1, 8])
def test_strided_results(pad):
    for m in (3, 40, 700):
        check(m, 136, 256, BF, bias=True, gate=2, residual=True, pad=pad)


def test_scales_past_a_vector():
    # more blocks along K than a wave has lanes
    for m in (16, 200):
        check(m, 64, 128 * 65 + 48)
        check(m, 64, 128 * 130)


def test_extreme_scales_and_lost_values():
    xq, xs, wq, ws, _ = operands(70, 96, 512)
    clean = bq.gemm_fp8(xq, xs, wq, ws)
    big = bq.gemm_fp8(xq, xs * 2.0 ** 60, wq, ws * 2.0 ** -60)
    assert torch.equal(big, clean)
    xq8 = xq.view(torch.uint8)
    xq8[5, 300] = 0x7F                       # NaN
    y = bq.gemm_fp8(xq, xs, wq, ws)
    keep = [i for i in range(70) if i != 5]
    assert y[5].isnan().all() and torch.equal(y[keep], clean[keep])
    xs = xs.clone()
    xq8[5, 300] = 0
    xs[2, 9] = math.inf
    y = bq.gemm_fp8(xq, xs, wq, ws)
    keep = [i for i in range(70) if i not in (5, 9)]
    assert not y[9].isfinite().any() and torch.equal(y[keep], clean[keep])
    zero = bq.gemm_fp8(torch.zeros_like(xq8).view(F8), xs.clamp(max=1.0), wq, ws)
    assert (zero == 0).all()


@pytest.mark.parametrize("m,k,n", [(1, 16, 40), (20, 144, 130), (333, 1552, 264)])
def test_linear_is_quantize_and_gemm(m, k, n):
    g = torch.Generator().manual_seed(k)
    for dtype in (BF, HF):
        x = (torch.randn(m, k + 3, generator=g) * 2).to(dtype).cuda()[:, :k]
        wq, ws = bq.pack_fp8((torch.randn(n, k, generator=g) * k ** -0.5).to(dtype))
        wq, ws = wq.cuda(), ws.cuda()
        b, r = torch.randn(n, generator=g).to(dtype).cuda(), torch.randn(m, n, generator=g).to(dtype).cuda()
        y = bq.linear_fp8(x, wq, ws, b, activation="silu", residual=r)
        assert torch.equal(y, bq.gemm_fp8(*bq.quantize_fp8(x), wq, ws, b, dtype=dtype, activation="silu", residual=r))
        want = bq.gemm_fp8(*bq.quantize_fp8(x), wq, ws, dtype=dtype, residual=r)
        assert torch.equal(bq.linear_fp8(x, wq, ws, residual=r, out=r), want)   # out may be residual
        assert bq.linear_fp8(x[:0], wq, ws).shape == (0, n)


def test_stream_graph_and_repeat():
    for m, n, k in ((4, 512, 1024), (100, 256, 8192), (600, 2048, 1024)):
        xq, xs, wq, ws, _ = operands(m, n, k)
        want = bq.gemm_fp8(xq, xs, wq, ws)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = [bq.gemm_fp8(xq, xs, wq, ws) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(y, want) for y in got)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            static = bq.gemm_fp8(xq, xs, wq, ws)
        for i in range(3):
            xs.mul_(1.5)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(static, bq.gemm_fp8(xq, xs, wq, ws))


def test_refuses():
    xq, xs, wq, ws, _ = operands(4, 32, 64)
    bf = torch.zeros(32, dtype=BF, device="cuda")
    for call in (lambda: bq.gemm_fp8(xq.float(), xs, wq, ws), lambda: bq.gemm_fp8(xq, xs.half(), wq, ws), lambda: bq.gemm_fp8(xq, xs, wq.cpu(), ws),
                 lambda: bq.gemm_fp8(xq, xs, wq, ws.double()), lambda: bq.gemm_fp8(xq, xs, wq, ws, bf.half()), lambda: bq.gemm_fp8(None, xs, wq, ws),
                 lambda: bq.linear_fp8(xq, wq, ws), lambda: bq.gemm_fp8(xq, xs, wq, None)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: bq.gemm_fp8(xq, xs[:, :3], wq, ws), lambda: bq.gemm_fp8(xq, xs, wq[:, :48], ws), lambda: bq.gemm_fp8(xq, xs, wq, ws, bf[:31]),
                 lambda: bq.gemm_fp8(xq, xs, wq, ws, dtype=torch.float32), lambda: bq.gemm_fp8(xq, xs, wq, ws, activation="relu"),
                 lambda: bq.gemm_fp8(xq.t().contiguous().t(), xs, wq, ws), lambda: bq.gemm_fp8(xq, xs, wq, ws, out=torch.zeros(4, 31, dtype=BF, device="cuda")),
                 lambda: bq.gemm_fp8(xq, xs, wq, ws, gate=torch.zeros(3, 32, dtype=BF, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros(4, 24, dtype=torch.uint8, device="cuda").view(F8)
    with pytest.raises(bq.SvdqError):
        bq.gemm_fp8(odd, xs, torch.zeros(32, 24, dtype=torch.uint8, device="cuda").view(F8), ws)
    off = torch.zeros(4 * 64 + 8, dtype=torch.uint8, device="cuda")[8:].view(4, 64).view(F8)
    with pytest.raises(bq.SvdqError):
        bq.gemm_fp8(off, xs, wq, ws)
