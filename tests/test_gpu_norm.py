"""GPU parity of the adaptive layer norm against a plain 64-bit reference."""

import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import assert_within, layer_norm_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def check(m, k, dtype, affine=False, groups=0, group_rows=None, pad=0, mean=0.0, std=1.0, eps=1e-6, x=None):
    print("layer_norm", m, k, dtype, affine, groups, pad, mean, std, flush=True)
    g = torch.Generator().manual_seed(m + k)

    def mat(r, c, s=1.0, b=0.0):
        return (torch.randn(r, c + pad, generator=g) * s + b).to(dtype).cuda()[:, :c]

    x = mat(m, k, std, mean) if x is None else x
    w, b = (mat(1, k, 0.2, 1.0)[0], mat(1, k)[0]) if affine else (None, None)
    sc, sh = (mat(groups, k, 0.3), mat(groups, k)) if groups else (None, None)
    out = None
    if pad:
        whole = torch.full((m, k + pad), 5.0, dtype=dtype, device="cuda")
        out = whole[:, :k]
    y = bq.layer_norm(x, w, b, scale=sc, shift=sh, group_rows=group_rows, eps=eps, out=out)
    torch.cuda.synchronize()
    if pad:
        assert (whole[:, k:] == 5).all()
    want, bound = layer_norm_reference(x, w, b, sc, sh, group_rows or (m // groups if groups else 1), eps)
    assert_within(y, want, bound, f"{m}x{k}")


# around every switch of the row's layout, odd sizes among them
@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 15, 63, 64, 65, 72, 127, 128, 129, 255, 256, 257, 260, 511, 512, 513, 520, 1023, 1024, 1031,
                               2048, 2049, 2056, 3072, 3073, 3080, 4095, 4096, 4097, 4104, 8192, 8193, 8200, 12288, 16384, 16385, 16392,
                               40000, 65535, 65536])
def test_widths(k):
    for dtype in (BF, HF):
        check(3, k, dtype)
        check(5, k, dtype, affine=True, groups=1)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 31, 33, 257, 1000])
@pytest.mark.parametrize("k", [40, 200, 768, 3072])
def test_rows_and_groups(m, k):
    check(m, k, BF, groups=m)
    check(m, k, HF, groups=-(-m // 3), group_rows=3)
    check(m, k, BF, affine=True)


@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strided_and_misaligned(pad):
    for k in (64, 77, 1000, 5000):
        check(9, k, BF, affine=True, groups=3, pad=pad)
        check(9, k, HF, pad=pad)


def test_off_centre_constant_and_extreme_rows():
    for k in (100, 3072, 9000):
        check(4, k, HF, mean=500.0, std=1.0)
        check(4, k, BF, mean=-300.0, std=4.0)
        check(4, k, BF, std=1e15)
        check(4, k, BF, std=1e-18, eps=0.0)
        check(4, k, BF, x=torch.full((4, k), 3.0, dtype=BF, device="cuda"))   # no variance: eps alone
    x = torch.randn(6, 3072, device="cuda").to(BF)
    clean = bq.layer_norm(x)
    x[2, 5], x[4, 9] = math.nan, math.inf
    y = bq.layer_norm(x)
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], clean[keep]) and y[2].isnan().all() and y[4].isnan().all()


def test_parts_of_the_modulation_and_in_place():
    x = torch.randn(10, 520, device="cuda").to(BF)
    v = [torch.randn(520, device="cuda").to(BF) for _ in range(4)]
    for i in range(4):
        kw = dict(zip(("weight", "bias", "scale", "shift"), (t if j == i else None for j, t in enumerate(v))))
        y = bq.layer_norm(x, kw["weight"], kw["bias"], scale=kw["scale"], shift=kw["shift"])
        want, bound = layer_norm_reference(x, kw["weight"], kw["bias"], kw["scale"], kw["shift"], 1, 1e-6)
        assert_within(y, want, bound, str(i))
    want = bq.layer_norm(x, v[0], v[1])
    assert torch.equal(bq.layer_norm(x, v[0], v[1], out=x), want)
    # modulation read in place out of one projection's output, as [groups][6 K]
    x = torch.randn(8, 256, device="cuda").to(HF)
    m = torch.randn(2, 6 * 256, device="cuda").to(HF)
    y = bq.layer_norm(x, scale=m[:, 256:512], shift=m[:, :256])
    want, bound = layer_norm_reference(x, None, None, m[:, 256:512], m[:, :256], 4, 1e-6)
    assert_within(y, want, bound, "in place")


def test_far_rows_and_empty():
    ld, m = 2 ** 25, 70
    buf = torch.empty(ld * m, dtype=BF, device="cuda")
    x = buf.as_strided((m, 200), (ld, 1))
    x.copy_(torch.randn(m, 200))
    check(m, 200, BF, x=x)
    assert bq.layer_norm(x[:0]).shape == (0, 200)


def test_stream_and_graph():
    x = torch.randn(64, 3072, device="cuda").to(BF)
    want = bq.layer_norm(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = bq.layer_norm(x)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = bq.layer_norm(x)
    keep = x.clone()
    for i in range(3):
        x.copy_(keep + i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, bq.layer_norm(x))


def test_wrapper_refuses():
    x = torch.zeros(4, 64, device="cuda", dtype=BF)
    with pytest.raises(TypeError):
        bq.layer_norm(x.float())
    with pytest.raises(TypeError):
        bq.layer_norm(x, torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        bq.layer_norm(x, torch.ones(63, device="cuda", dtype=BF))
    with pytest.raises(ValueError):
        bq.layer_norm(x, scale=torch.ones(3, 64, device="cuda", dtype=BF))
    with pytest.raises(ValueError):
        bq.layer_norm(x, scale=torch.ones(4, 64, device="cuda", dtype=BF), shift=torch.ones(2, 64, device="cuda", dtype=BF))
    with pytest.raises(bq.SvdqError):
        bq.layer_norm(x, eps=-1.0)
    with pytest.raises(bq.SvdqError):
        bq.layer_norm(torch.zeros(1, 65537, device="cuda", dtype=BF))


def test_more_rows_than_one_axis_of_a_launch():
    m, k = 2 ** 29 + 5, 8   # 8 lanes a row: past 2^32 threads, and past 2^32 elements
    g = torch.Generator().manual_seed(8)
    part = torch.randn(2 ** 20, k, generator=g).to(BF).cuda()
    x = torch.empty(m, k, dtype=BF, device="cuda")
    x[:2 ** 29].view(2 ** 9, 2 ** 20, k).copy_(part.expand(2 ** 9, -1, -1))
    x[2 ** 29:] = part[:5]
    y = bq.layer_norm(x, out=x)
    torch.cuda.synchronize()
    want, bound = layer_norm_reference(part, None, None, None, None, 1, 1e-6)
    for first in (0, 2 ** 20, 2 ** 24 - 2 ** 20, 2 ** 28, 2 ** 29 - 2 ** 20):
        assert_within(y[first:first + 2 ** 20], want, bound, f"rows from {first}")
    assert_within(y[2 ** 29:], want[:5], bound[:5] if torch.is_tensor(bound) else bound, "last rows")
