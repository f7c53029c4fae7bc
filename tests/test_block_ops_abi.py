"""The 16-bit operators' C entry points refuse bad arguments before anything
is launched."""

import ctypes
import math

import pytest
import torch

import bit_quantized_diffusion_amd as bq

FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced (validation fails first)
MIS = ctypes.c_void_p(0x10004)       # misaligned
ODD = ctypes.c_void_p(0x10002)
BAD, SHAPE = bq.SVDQ_ERR_INVALID_ARG, bq.SVDQ_ERR_SHAPE


def _gpu_present():
    import torch
    return torch.cuda.is_available()


ATTENTION = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=None, cu_q=FAKE, cu_k=FAKE, batch=2, tq=10, tk=20, hq=4, hk=2, d=64,
                 strides=(256, 64, 128, 64, 128, 64, 256, 64), scale=0.125, causal=0, dtype=0, ws=None, n=0)


def attention(**kw):
    a = dict(ATTENTION, **kw)
    strides = None if a["strides"] is None else (ctypes.c_int64 * 8)(*a["strides"])
    return bq.lib.svdq_attention(a["q"], a["k"], a["v"], a["o"], a["lse"], a["cu_q"], a["cu_k"], a["batch"], a["tq"], a["tk"],
                                 a["hq"], a["hk"], a["d"], strides, a["scale"], a["causal"], a["dtype"], a["ws"], a["n"], None)


def with_stride(i, value):
    s = list(ATTENTION["strides"])
    s[i] = value
    return tuple(s)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(o=None), BAD), (dict(q=MIS), BAD), (dict(k=MIS), BAD),
    (dict(v=MIS), BAD), (dict(o=MIS), BAD), (dict(ws=MIS), BAD), (dict(lse=ODD), BAD), (dict(cu_q=ODD), BAD),
    (dict(cu_q=None), BAD), (dict(cu_k=None), BAD), (dict(cu_q=None, cu_k=None), BAD), (dict(strides=None), BAD),
    (dict(strides=with_stride(0, 252)), BAD), (dict(strides=with_stride(3, -64)), BAD), (dict(strides=with_stride(2, 56)), BAD),
    (dict(strides=with_stride(4, (1 << 23) + 8)), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD), (dict(dtype=2), BAD),
    (dict(batch=0), SHAPE), (dict(tq=-1), SHAPE), (dict(tk=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hk=3), SHAPE), (dict(hk=0), SHAPE),
    (dict(d=0), SHAPE), (dict(d=60), SHAPE), (dict(d=136), SHAPE), (dict(tq=2 ** 31 - 1, hq=64, hk=2), SHAPE),
    (dict(tq=2 ** 30, hq=64, hk=64), SHAPE), (dict(tk=2 ** 31 - 100), SHAPE), (dict(tq=2 ** 31 - 100, hq=1, hk=1), SHAPE),
    (dict(scale=3e38), BAD), (dict(tq=2 ** 29, hq=1, hk=1), SHAPE), (dict(batch=2 ** 24), SHAPE),
])
def test_attention_refuses(kw, want):
    assert attention(**kw) == want


def test_attention_workspace_size():
    f = bq.lib.svdq_attention_workspace_size
    out = ctypes.c_size_t(7)
    assert f(1, 1, 1, 1, 1, 64, None) == BAD
    assert f(1, 1, 1, 3, 2, 64, ctypes.byref(out)) == SHAPE and out.value == 0
    assert bq.attention_workspace_size(4608, 4608, 1, 24, 24, 128) == 0
    assert bq.attention_workspace_size(1, 8192, 1, 8, 8, 128) > 0      # one token against a long cache


@pytest.mark.skipif(_gpu_present(), reason="checks the no-device path")
def test_no_device():
    assert attention() == bq.SVDQ_ERR_UNSUPPORTED_DEVICE


LINEAR = dict(x=FAKE, ldx=64, w=FAKE, ldw=64, bias=FAKE, gate=FAKE, ld_gate=32, rows=4, residual=FAKE, ldr=32, y=FAKE, ldy=32,
              m=8, n=32, k=64, act=0, dtype=0, ws=None, size=0)
NORM = dict(x=FAKE, ldx=64, weight=FAKE, bias=FAKE, scale=FAKE, shift=FAKE, ld=64, rows=4, y=FAKE, ldy=64, m=8, k=64, eps=1e-6,
            dtype=0)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(x=ctypes.c_void_p(0x10001)), BAD),
    (dict(residual=ctypes.c_void_p(0x10001)), BAD), (dict(ws=MIS), BAD), (dict(act=3), BAD), (dict(dtype=-1), BAD),
    (dict(m=0), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(ldx=63), SHAPE), (dict(ldw=63), SHAPE), (dict(ldy=31), SHAPE),
    (dict(ldr=31), SHAPE), (dict(ld_gate=31), SHAPE), (dict(rows=0), SHAPE), (dict(ldx=(1 << 22) + 1), SHAPE),
    (dict(k=1 << 22, ldx=1 << 22, ldw=1 << 22), SHAPE), (dict(m=2 ** 31 - 100), SHAPE), (dict(n=2 ** 31 - 100, ldy=2 ** 31, ldr=2 ** 31, ld_gate=2 ** 31), SHAPE),
    (dict(n=2 ** 29, ldy=2 ** 29, ldr=2 ** 29, ld_gate=2 ** 29), SHAPE), (dict(m=2 ** 29, n=128, ldy=128, ldr=128, ld_gate=128), SHAPE),
])
def test_linear16_refuses(kw, want):
    assert bq.lib.svdq_linear16(*dict(LINEAR, **kw).values(), None) == want


def test_linear16_workspace_size():
    f = bq.lib.svdq_linear16_workspace_size
    out = ctypes.c_size_t(7)
    assert f(1, 1, 1, None) == BAD
    assert f(0, 1, 1, ctypes.byref(out)) == SHAPE and out.value == 0
    assert bq.linear16_workspace_size(4608, 12288, 3072) == 0
    assert bq.linear16_workspace_size(100, 256, 4096) % (100 * 256 * 4) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(scale=ctypes.c_void_p(0x10001)), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD), (dict(dtype=5), BAD), (dict(m=0), SHAPE), (dict(k=0), SHAPE),
    (dict(k=65537, ldx=65537, ldy=65537, ld=65537), SHAPE), (dict(ldx=63), SHAPE), (dict(ldy=63), SHAPE), (dict(ld=63), SHAPE),
    (dict(rows=0), SHAPE), (dict(m=2 ** 31 - 100), SHAPE),
])
def test_layer_norm_refuses(kw, want):
    assert bq.lib.svdq_layer_norm(*dict(NORM, **kw).values(), None) == want


@pytest.mark.skipif(_gpu_present(), reason="checks the no-device path")
def test_no_device_linear16_and_norm():
    assert bq.lib.svdq_linear16(*LINEAR.values(), None) == bq.SVDQ_ERR_UNSUPPORTED_DEVICE
    assert bq.lib.svdq_layer_norm(*NORM.values(), None) == bq.SVDQ_ERR_UNSUPPORTED_DEVICE


def test_host_tensors_are_refused():
    x, w, q = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(16, 8, dtype=torch.bfloat16), torch.zeros(4, 2, 8, dtype=torch.float16)
    for call in (lambda: bq.linear16(x, w), lambda: bq.layer_norm(x), lambda: bq.attention(q, q, q), lambda: bq.layer_norm([1.0]),
                 lambda: bq.linear16(x.float(), w), lambda: bq.attention(None, q, q)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        bq.linear16(x, w, activation="relu")


def test_linear16_workspace_size_for_operands():
    """The plan goes by the operands' alignment; the query without them names
    enough for either."""
    f = bq.lib.svdq_linear16_workspace_size_for
    out = ctypes.c_size_t(7)

    def named(x, ldx, w, ldw, m, n, k):
        assert f(x, ldx, w, ldw, m, n, k, ctypes.byref(out)) == 0
        return out.value

    assert f(FAKE, 64, FAKE, 64, 1, 1, 64, None) == BAD
    assert f(FAKE, 64, FAKE, 64, 0, 1, 64, ctypes.byref(out)) == SHAPE and out.value == 0
    for m, n, k in ((16, 64, 15360), (1, 32, 8192), (32, 512, 4096)):   # up to 32 rows: only misaligned ones are split
        assert named(FAKE, k, FAKE, k, m, n, k) == 0
        for args in ((ODD, k, FAKE, k), (FAKE, k, ODD, k), (FAKE, k + 1, FAKE, k), (FAKE, k, FAKE, k + 4)):
            assert 0 < named(*args, m, n, k) <= bq.linear16_workspace_size(m, n, k)
    for m, n, k in ((100, 256, 4096), (40, 130, 2056), (333, 512, 8192), (300, 33, 1024), (4608, 128, 15360)):
        most = max(named(FAKE, k, FAKE, k, m, n, k), named(ODD, k, FAKE, k, m, n, k))
        assert bq.linear16_workspace_size(m, n, k) == most
