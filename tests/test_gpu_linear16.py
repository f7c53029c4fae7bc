"""GPU parity of the 16-bit linear with its epilogue against a plain 64-bit
reference, element by element."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import assert_within, linear16_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def check(m, n, k, dtype=BF, act="none", bias=True, gate=0, residual=False, seed=0, pad=0, group_rows=None, **kw):
    """`pad`: elements between the rows of every matrix (odd ones misalign them)."""
    print("linear16", m, n, k, dtype, act, bias, gate, residual, pad, flush=True)
    g = torch.Generator().manual_seed(seed + m + n + k)

    def mat(r, c, std=1.0):
        return (torch.randn(r, c + pad, generator=g) * std).to(dtype).cuda()[:, :c]

    x, w = mat(m, k), mat(n, k, k ** -0.5)
    b = mat(1, n, 0.5)[0] if bias else None
    gt = mat(gate, n) if gate else None
    r = mat(m, n) if residual else None
    rows = group_rows or (m // gate if gate else None)
    out = None
    if pad:
        whole = torch.full((m, n + pad), 5.0, dtype=dtype, device="cuda")
        out = whole[:, :n]
    y = bq.linear16(x, w, b, activation=act, gate=gt, residual=r, group_rows=group_rows, out=out, **kw)
    torch.cuda.synchronize()
    if pad:
        assert (whole[:, n:] == 5).all()
    want, bound = linear16_reference(x, w, b, act, gt, r, rows)
    assert_within(y, want, bound, f"{m}x{n}x{k}")
    return y


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32])
@pytest.mark.parametrize("n,k", [(64, 128), (33, 8), (200, 1000), (1, 264), (96, 4096)])
def test_few_rows(m, n, k):
    check(m, n, k, BF if m % 2 else HF, act="silu" if m % 3 else "none")


@pytest.mark.parametrize("m", [1, 7, 9, 13, 16, 17, 30, 32])
def test_few_rows_many_channels(m):
    """More workgroups than CUs: two waves each from 9 rows on."""
    check(m, 8500, 200, act="gelu", gate=1, residual=True)


@pytest.mark.parametrize("m,n,k", [(33, 128, 64), (64, 64, 72), (127, 129, 200), (128, 128, 8), (129, 257, 1024), (333, 520, 136),
                                   (300, 40, 16), (40, 1, 64), (513, 130, 2048)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_middle(m, n, k, dtype):
    check(m, n, k, dtype, act="gelu", residual=True)
    check(m, n, k, dtype, gate=1)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 7, 3), (2, 33, 65), (5, 100, 127), (33, 17, 9), (130, 131, 133), (64, 64, 63), (200, 65, 1023)])
@pytest.mark.parametrize("pad", [0, 1, 3])
def test_odd_and_misaligned(m, n, k, pad):
    for dtype in (BF, HF):
        check(m, n, k, dtype, act="silu", gate=1, residual=True, pad=pad)


def test_padded_rows_stay_on_the_fast_path():
    for m in (3, 100):
        check(m, 72, 128, pad=8, residual=True, gate=1)
        check(m, 72, 120, pad=8)


@pytest.mark.parametrize("m,n,k", [(3072, 4096, 200), (2900, 4333, 64), (4608, 3072, 264)])
def test_large_tiles(m, n, k):
    check(m, n, k, BF, act="gelu", residual=True, gate=4 if m % 4 == 0 else 1)


def test_split_along_k():
    for m, n, k, split in ((100, 256, 4096, True), (40, 130, 2048 + 8, True), (300, 33, 1024, False)):
        assert (bq.linear16_workspace_size(m, n, k) > 0) == split
        a = check(m, n, k, act="gelu", residual=True, gate=2)
        b = check(m, n, k, act="gelu", residual=True, gate=2, workspace=None)
        assert torch.equal(a, check(m, n, k, act="gelu", residual=True, gate=2))
        assert a.shape == b.shape
    check(100, 131, 2049, act="gelu", residual=True)         # unaligned, split


@pytest.mark.parametrize("groups,rows", [(1, None), (2, None), (7, 5), (35, 1), (2, 34)])
def test_gate_groups(groups, rows):
    m = 35 if rows else 34
    check(m, 70, 64, gate=groups, group_rows=rows, residual=True)
    g = torch.randn(50, device="cuda").to(BF)
    x, w = torch.randn(4, 64, device="cuda").to(BF), torch.randn(50, 64, device="cuda").to(BF)
    assert torch.equal(bq.linear16(x, w, gate=g), bq.linear16(x, w, gate=g[None]))


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_wide_values_and_not_finite(act):
    """Arguments far into both tails of the activations; a NaN or infinity
    stays in its row."""
    x = torch.zeros(40, 64, dtype=BF, device="cuda")
    x[:, 0] = torch.linspace(-300, 300, 40, device="cuda").to(BF)
    w = torch.zeros(8, 64, dtype=BF, device="cuda")
    w[:, 0] = 1
    y = bq.linear16(x, w, activation=act)
    want, bound = linear16_reference(x, w, None, act, None, None, None)
    assert_within(y, want, bound, act)
    clean = bq.linear16(x[:20], w, activation=act)
    x[5, 3] = math.nan
    x[7, 0] = math.inf
    for n in (40, 20):
        y = bq.linear16(x[:n].contiguous(), w, activation=act)
        assert y[5].isnan().all() and (y[7] == math.inf).all()
        keep = [i for i in range(20) if i not in (5, 7)]
        assert torch.equal(y[keep], clean[keep])


def test_residual_in_place():
    for m, n, k in ((3, 96, 256), (200, 130, 64), (200, 130, 4096)):
        x, w = torch.randn(m, k, device="cuda").to(BF), (torch.randn(n, k, device="cuda") * k ** -0.5).to(BF)
        r = torch.randn(m, n, device="cuda").to(BF)
        want = bq.linear16(x, w, residual=r)
        got = r.clone()
        assert bq.linear16(x, w, residual=got, out=got) is got
        assert torch.equal(got, want)


def test_far_rows():
    """Row strides with which a tile's rows lie megabytes, the whole operand
    gigabytes apart."""
    ld, m, k = 2 ** 22, 300, 72
    buf = torch.empty(ld * m, dtype=BF, device="cuda")
    x = buf.as_strided((m, k), (ld, 1))
    x.copy_(torch.randn(m, k))
    w = torch.randn(40, k, device="cuda").to(BF)
    for a, b in ((x, w), (w, x), (x[:20], w)):
        y = bq.linear16(a, b)
        want, bound = linear16_reference(a, b, None, "none", None, None, None)
        assert_within(y, want, bound, "far rows")


def test_empty_stream_and_graph():
    x, w = torch.randn(150, 2048, device="cuda").to(BF), torch.randn(64, 2048, device="cuda").to(BF)
    assert bq.linear16(x[:0], w).shape == (0, 64)
    want = bq.linear16(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = bq.linear16(x, w)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = bq.linear16(x, w)
    keep = x.clone()
    for i in range(3):
        x.copy_(keep * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, bq.linear16(x, w))


def test_wrapper_refuses():
    x, w = torch.zeros(4, 64, device="cuda", dtype=BF), torch.zeros(8, 64, device="cuda", dtype=BF)
    with pytest.raises(TypeError):
        bq.linear16(x.float(), w.float())
    with pytest.raises(TypeError):
        bq.linear16(x, w.half())
    with pytest.raises(ValueError):
        bq.linear16(x, w[:, :32])
    with pytest.raises(ValueError):
        bq.linear16(x, w, activation="relu6")
    with pytest.raises(ValueError):
        bq.linear16(x, w, torch.zeros(7, device="cuda", dtype=BF))
    with pytest.raises(ValueError):
        bq.linear16(x, w, gate=torch.zeros(3, 8, device="cuda", dtype=BF))
    with pytest.raises(ValueError):
        bq.linear16(x, w, gate=torch.zeros(2, 8, device="cuda", dtype=BF), group_rows=1)
    with pytest.raises(ValueError):
        bq.linear16(x.t(), w)
    with pytest.raises(ValueError):
        bq.linear16(x, w, residual=torch.zeros(4, 9, device="cuda", dtype=BF))
