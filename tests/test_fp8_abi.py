"""The 8-bit operators on the host: their C entry points refuse bad arguments
before anything is launched, and the weight's pack follows its rule."""

import ctypes
import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference8 import pack_plain

FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced (validation fails first)
OFF = ctypes.c_void_p(0x10008)       # 8-byte aligned
ODD = ctypes.c_void_p(0x10001)
BAD, SHAPE = bq.SVDQ_ERR_INVALID_ARG, bq.SVDQ_ERR_SHAPE


def _gpu_present():
    return torch.cuda.is_available()


NORM = dict(x=FAKE, ldx=64, residual=FAKE, ldr=64, weight=FAKE, sum=FAKE, ld_sum=64, y=FAKE, ldy=64, yq=None, ys=None, m=8, k=64,
            eps=1e-6, dtype=0)
CODES = dict(NORM, y=None, yq=FAKE, ys=FAKE)
QUANT = dict(x=FAKE, ldx=64, xq=FAKE, xs=FAKE, m=8, k=64, dtype=0)
GEMM = dict(xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, bias=FAKE, gate=FAKE, ld_gate=32, rows=4, residual=FAKE, ldr=32, y=FAKE, ldy=32, m=8,
            n=32, k=64, act=0, dtype=0)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(yq=FAKE, ys=FAKE), BAD), (dict(x=ODD), BAD), (dict(residual=ODD), BAD), (dict(sum=ODD), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD), (dict(dtype=2), BAD), (dict(m=0), SHAPE), (dict(k=0), SHAPE),
    (dict(m=2 ** 31 - 100), SHAPE), (dict(k=65537, ldx=65537, ldr=65537, ld_sum=65537, ldy=65537), SHAPE), (dict(ldx=63), SHAPE),
    (dict(ldr=63), SHAPE), (dict(ld_sum=63), SHAPE), (dict(ldy=63), SHAPE),
])
def test_rms_norm_refuses(kw, want):
    assert bq.lib.svdq_rms_norm(*dict(NORM, **kw).values(), None) == want


@pytest.mark.parametrize("kw,want", [(dict(ys=None), BAD), (dict(yq=None), BAD), (dict(yq=OFF), BAD), (dict(ys=ODD), BAD), (dict(k=40), SHAPE)])
def test_rms_norm_codes_refuses(kw, want):
    assert bq.lib.svdq_rms_norm(*dict(CODES, **kw).values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(xq=None), BAD), (dict(xs=None), BAD), (dict(x=ODD), BAD), (dict(xq=OFF), BAD), (dict(xs=ODD), BAD), (dict(dtype=9), BAD),
    (dict(m=0), SHAPE), (dict(k=0), SHAPE), (dict(k=8), SHAPE), (dict(k=72), SHAPE), (dict(ldx=63), SHAPE), (dict(k=(1 << 22) + 16, ldx=1 << 23), SHAPE),
])
def test_quantize_refuses(kw, want):
    assert bq.lib.svdq_quantize_fp8(*dict(QUANT, **kw).values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(xq=None), BAD), (dict(xs=None), BAD), (dict(wq=None), BAD), (dict(ws=None), BAD), (dict(y=None), BAD), (dict(xq=OFF), BAD),
    (dict(wq=OFF), BAD), (dict(xs=ODD), BAD), (dict(ws=ODD), BAD), (dict(y=ODD), BAD), (dict(residual=ODD), BAD),
    (dict(act=3), BAD), (dict(dtype=-1), BAD), (dict(m=0), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(k=72), SHAPE),
    (dict(k=(1 << 22) + 16), SHAPE), (dict(ldy=31), SHAPE), (dict(ldr=31), SHAPE), (dict(ld_gate=31), SHAPE), (dict(rows=0), SHAPE),
    (dict(m=2 ** 31 - 100), SHAPE), (dict(n=2 ** 28, ldy=2 ** 28, ldr=2 ** 28, ld_gate=2 ** 28), SHAPE),
    (dict(m=2 ** 28, n=128, ldy=128, ldr=128, ld_gate=128), SHAPE), (dict(m=2 ** 29, n=16, ldy=16, ldr=16, ld_gate=16), SHAPE),
])
def test_gemm_refuses(kw, want):
    assert bq.lib.svdq_gemm_fp8(*dict(GEMM, **kw).values(), None) == want


def test_plan_refuses():
    plan = (ctypes.c_int32 * 3)()
    assert bq.lib.svdq_debug_gemm_fp8_plan(1, 1, 16, None) == BAD
    assert bq.lib.svdq_debug_gemm_fp8_plan(0, 1, 16, plan) == SHAPE and bq.lib.svdq_debug_gemm_fp8_plan(1, 1, 24, plan) == SHAPE


def test_gemm_sizes_reach_every_tile_shape():
    from tests import test_gpu_gemm_fp8 as gemm
    for case, want in gemm.SHAPES.items():
        assert gemm.plan(*case) == want, case
    assert len(set(gemm.SHAPES.values())) == len(gemm.SHAPES) == 14


@pytest.mark.skipif(_gpu_present(), reason="checks the no-device path")
def test_no_device():
    for call in (lambda: bq.lib.svdq_rms_norm(*NORM.values(), None), lambda: bq.lib.svdq_rms_norm(*CODES.values(), None),
                 lambda: bq.lib.svdq_quantize_fp8(*QUANT.values(), None), lambda: bq.lib.svdq_gemm_fp8(*GEMM.values(), None)):
        assert call() == bq.SVDQ_ERR_UNSUPPORTED_DEVICE


def test_host_tensors_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, s = torch.zeros(16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(1, 1)
    for call in (lambda: bq.rms_norm(x), lambda: bq.rms_norm_fp8(x), lambda: bq.quantize_fp8(x), lambda: bq.linear_fp8(x, w, s),
                 lambda: bq.gemm_fp8(w, s, w, s), lambda: bq.rms_norm([1.0]), lambda: bq.gemm_fp8(None, s, w, s)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("n,k", [(1, 16), (128, 128), (130, 272), (300, 1040)])
def test_pack(n, k):
    g = torch.Generator().manual_seed(n)
    for dtype in (torch.bfloat16, torch.float16):
        w = (torch.randn(n, k, generator=g) * torch.exp(torch.randn(n, k, generator=g) * 2)).to(dtype)
        w[0, :3] = torch.tensor([0.0, -0.0, 5.0]).to(dtype)
        q, s = bq.pack_fp8(w)
        want_q, want_s = pack_plain(w)
        assert torch.equal(s, want_s)
        assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8))


def test_pack_of_every_step():
    """Values that meet every code, and the middle between two of them."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    w = torch.cat([codes, (codes[1:] + codes[:-1]) / 2, -codes, torch.tensor([448.0])])
    w = torch.nn.functional.pad(w, (0, 512 - w.numel())).view(4, 128).to(torch.bfloat16)   # the largest, 448: scale 1
    assert w.float().abs().max() == 448
    q, s = bq.pack_fp8(w)
    assert (s == 1).all()
    assert torch.equal(q.view(torch.uint8), w.float().to(torch.float8_e4m3fn).view(torch.uint8))


def test_pack_refuses():
    for w in (torch.zeros(4, 16), torch.zeros(4, dtype=torch.bfloat16), None):
        with pytest.raises(TypeError):
            bq.pack_fp8(w)
    for w in (torch.zeros(4, 24, dtype=torch.bfloat16), torch.zeros(0, 16, dtype=torch.float16)):
        with pytest.raises(bq.SvdqError):
            bq.pack_fp8(w)


APPEND = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, strides=(256, 64, 128, 64, 128, 64, 256, 64), k8=FAKE, v8=FAKE, e=FAKE, pages=4, table=FAKE,
              width=2, lengths=FAKE, cu=FAKE, batch=2, total=10, hq=4, hk=2, d=64, rope=FAKE, rows=128, rotary=64, interleaved=0, dtype=0)
PAGED = dict(q=FAKE, o=FAKE, lse=FAKE, strides=(256, 64, 256, 64), k8=FAKE, v8=FAKE, e=FAKE, pages=4, table=FAKE, width=2, lengths=FAKE, cu=FAKE,
             batch=2, total=10, hq=4, hk=2, d=64, scale=0.125, causal=1, dtype=0, ws=None, n=0)


def _call(fn, defaults, kw):
    a = dict(defaults, **kw)
    a["strides"] = None if a["strides"] is None else (ctypes.c_int64 * len(a["strides"]))(*a["strides"])
    return fn(*a.values(), None)


SHAPES = [
    (dict(batch=0), SHAPE), (dict(total=-1), SHAPE), (dict(width=0), SHAPE), (dict(hq=0), SHAPE), (dict(hk=0), SHAPE), (dict(hk=3), SHAPE),
    (dict(pages=0), SHAPE), (dict(d=8), SHAPE), (dict(d=72), SHAPE), (dict(d=144), SHAPE), (dict(cu=None), SHAPE), (dict(total=2 ** 24), SHAPE),
    (dict(batch=2 ** 23), SHAPE), (dict(width=2 ** 30), SHAPE), (dict(width=2 ** 24 + 1, hq=1, hk=1, batch=1, total=1), SHAPE), (dict(total=2 ** 23, hq=512), SHAPE),
    (dict(k8=None), BAD), (dict(v8=None), BAD), (dict(e=None), BAD), (dict(table=None), BAD), (dict(lengths=None), BAD), (dict(strides=None), BAD),
    (dict(k8=OFF), BAD), (dict(v8=OFF), BAD), (dict(table=ODD), BAD), (dict(lengths=ODD), BAD), (dict(cu=ODD), BAD), (dict(dtype=2), BAD),
]


@pytest.mark.parametrize("kw,want", SHAPES + [
    (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=ODD), BAD), (dict(q_out=ODD), BAD), (dict(rope=ODD), BAD),
    (dict(strides=(256, 64, -128, 64, 128, 64, 256, 64)), BAD), (dict(strides=(256, 64, 128, 64, 128, 64, 1 << 41, 64)), BAD),
    (dict(rotary=0), SHAPE), (dict(rope=None), SHAPE), (dict(rotary=24), SHAPE), (dict(rotary=80), SHAPE), (dict(rotary=-16), SHAPE), (dict(rows=0), SHAPE),
])
def test_append_refuses(kw, want):
    assert _call(bq.lib.svdq_cache_append, APPEND, kw) == want


@pytest.mark.parametrize("kw,want", SHAPES + [
    (dict(q=None), BAD), (dict(o=None), BAD), (dict(q=OFF), BAD), (dict(o=OFF), BAD), (dict(lse=ODD), BAD), (dict(ws=OFF), BAD), (dict(scale=0.0), BAD),
    (dict(scale=math.nan), BAD), (dict(scale=2.0 ** 80), BAD), (dict(scale=2.0 ** -81), BAD), (dict(strides=(256, 60, 256, 64)), BAD), (dict(strides=(256, 64, -256, 64)), BAD),
])
def test_attention_paged_refuses(kw, want):
    assert _call(bq.lib.svdq_attention_paged, PAGED, kw) == want


def test_paged_workspace_and_plan():
    out, plan = ctypes.c_size_t(7), (ctypes.c_int32 * 2)()
    f, g = bq.lib.svdq_attention_paged_workspace_size, bq.lib.svdq_debug_attention_paged_plan
    assert f(1, 1, 1, 1, 1, 64, None) == BAD and g(1, 1, 1, 1, 1, 64, None) == BAD
    assert f(1, 1, 1, 3, 2, 64, ctypes.byref(out)) == SHAPE and out.value == 0 and g(1, 0, 1, 1, 1, 64, plan) == SHAPE
    assert bq.attention_paged_workspace_size(1, 1, 256, 8, 2, 128) > 0 and bq.attention_paged_workspace_size(1, 1, 4, 8, 2, 128) == 0


def test_paged_sizes_reach_every_schedule():
    from tests import test_gpu_attention_paged as paged
    for new, lens, hq, hk, d, _ in paged.MANY:
        width = max(-(-n // bq.PAGE) for n in lens) + 2
        assert paged.plan(sum(new), len(new), width, hq, hk, d) == (256 if d > 64 else 128, 0), (new, lens)
    for args, want in (((8, 8, 30, 8, 2, 128), (16, 512)), ((8, 8, 16, 8, 2, 128), (16, 0)), ((40, 8, 30, 8, 2, 128), (32, 512)),
                       ((40, 8, 10, 8, 2, 128), (32, 0)), ((64, 1, 128, 32, 8, 128), (32, 512)), ((3050, 4, 127, 32, 8, 128), (256, 0))):
        assert paged.plan(*args) == want, args


@pytest.mark.skipif(_gpu_present(), reason="checks the no-device path")
def test_no_device_cache():
    assert _call(bq.lib.svdq_cache_append, APPEND, {}) == bq.SVDQ_ERR_UNSUPPORTED_DEVICE
    assert _call(bq.lib.svdq_attention_paged, PAGED, {}) == bq.SVDQ_ERR_UNSUPPORTED_DEVICE


def test_host_caches_are_refused():
    cache = bq.KVCache.allocate(2, 2, 32, device="cpu")
    k, n = torch.zeros(1, 2, 32, dtype=torch.bfloat16), torch.ones(1, dtype=torch.int32)
    for call in (lambda: bq.cache_append(cache, k, k, n[None], n), lambda: bq.attention_paged(k, cache, n[None], n)):
        with pytest.raises(TypeError):
            call()


def test_cache_layout_and_angles():
    """What `read` takes from where svdq.h says the codes lie."""
    cache = bq.KVCache.allocate(3, 2, 16, device="cpu")
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    one, two = 0x38, 0x40      # 1.0 and 2.0
    k[2, 1, 5, 7] = one
    v[0, 0, 37 // 4 % 4, 3, 37 // 16 * 4 + 37 % 4] = two
    cache.exponents[2, 1, 0], cache.exponents[0, 0, 1] = -3, 4
    keys, values = cache.read(torch.tensor([2, 0], dtype=torch.int32), 110)
    assert keys.shape == values.shape == (110, 2, 16)
    assert keys[5, 1, 7] == 0.125 and keys.count_nonzero() == 1
    assert values[64 + 37, 0, 3] == 32.0 and values.count_nonzero() == 1
    table = bq.rope_table(1 << 17, 64, device="cpu")
    p, i = 99999, 3
    angle = p * 10000.0 ** (-2 * i / 64)
    assert abs(float(table[p, i]) - math.cos(angle)) < 1e-7 and abs(float(table[p, 32 + i]) - math.sin(angle)) < 1e-7
