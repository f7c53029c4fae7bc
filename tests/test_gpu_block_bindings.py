"""The Python side of the 16-bit block operators: what it refuses, and that it
keeps and loses no reference."""

import gc
import sys

import pytest
import torch

import bit_quantized_diffusion_amd as bq

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _require_device():
    assert bq.device_check(0), "gfx950 device required for the GPU tests"


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("bad", [None, 3, "x", [1.0], object(), torch.Size([2, 8])])
def test_no_tensors(bad):
    x, w, q = z(4, 8), z(16, 8), z(4, 2, 8)
    with pytest.raises(TypeError):
        bq.linear16(bad, w)
    with pytest.raises(TypeError):
        bq.linear16(x, bad)
    with pytest.raises(TypeError):
        bq.layer_norm(bad)
    for i in range(3):
        with pytest.raises(TypeError):
            bq.attention(*[bad if j == i else q for j in range(3)])
    if bad is not None:
        with pytest.raises(TypeError):
            bq.linear16(x, w, bad)
        with pytest.raises(TypeError):
            bq.linear16(x, w, gate=bad)
        with pytest.raises(TypeError):
            bq.linear16(x, w, residual=bad)
        with pytest.raises(TypeError):
            bq.linear16(x, w, out=bad)
        with pytest.raises(TypeError):
            bq.layer_norm(x, scale=bad)
        with pytest.raises(TypeError):
            bq.attention(q, q, q, cu_seqlens_q=bad)


def test_wrong_tensors():
    x, w, q = z(4, 8), z(16, 8), z(4, 2, 8)
    sparse = torch.eye(8, dtype=BF, device="cuda").to_sparse()
    for t in (x.cpu(), x.float(), z(4, 8, 1), z(8), z(2, 2, 2, 2), sparse):
        with pytest.raises(TypeError):
            bq.layer_norm(t)
    with pytest.raises(ValueError):
        bq.layer_norm(z(8, 4).t())
    for t in (w.cpu(), w.half(), z(16, 8, 1), z(8)):
        with pytest.raises(TypeError):
            bq.linear16(x, t)
    for t in (z(16, 9), z(8, 16).t()):
        with pytest.raises(ValueError):
            bq.linear16(x, t)
    for kw in (dict(gate=z(15)), dict(gate=z(3, 16)), dict(gate=z(2, 16), group_rows=1), dict(gate=z(2, 16), group_rows=0),
               dict(gate=z(2, 16), group_rows=-1), dict(gate=z(0, 16)), dict(gate=z(1, 1, 16)), dict(residual=z(4, 15)),
               dict(out=z(5, 16)), dict(activation="relu"), dict(activation=1)):
        with pytest.raises(ValueError):
            bq.linear16(x, w, **kw)
    with pytest.raises(TypeError):
        bq.linear16(x, w, gate=z(2, 16), group_rows=1.5)
    with pytest.raises(TypeError):
        bq.layer_norm(x, eps="small")
    with pytest.raises(TypeError):
        bq.attention(q, q, q, scale="small")
    with pytest.raises(TypeError):
        bq.attention(q, q, z(4, 2, 8, 1)[..., 0].half())
    for k in (z(4, 2, 16), z(4, 2, 8).transpose(0, 2)):
        with pytest.raises(ValueError):
            bq.attention(q, k, k)
    i32 = dict(dtype=torch.int32)
    for cu in (torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, **i32), z(1, 2, dtype=torch.int32),
               z(4, dtype=torch.int32)[::2]):
        with pytest.raises(TypeError):
            bq.attention(q, q, q, cu_seqlens_q=cu)
    with pytest.raises(ValueError):
        bq.attention(q, q, q, cu_seqlens_q=z(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        bq.attention(q, q, q, cu_seqlens_q=z(2, dtype=torch.int32), cu_seqlens_k=z(3, dtype=torch.int32))
    for ws in ("none", "AUTO"):
        with pytest.raises(ValueError):
            bq.linear16(x, w, workspace=ws)
    for ws in (z(64), torch.zeros(64, dtype=torch.uint8), z(64, dtype=torch.uint8)[::2], 5):
        with pytest.raises(TypeError):
            bq.attention(q, q, q, workspace=ws)


def test_sizes_that_the_library_does_not_count():
    far = z(1, 8).expand(2 ** 31, 8)
    with pytest.raises(ValueError):
        bq.layer_norm(far, out=far)
    with pytest.raises(ValueError):
        bq.linear16(far, z(16, 8), out=far)
    with pytest.raises(ValueError):
        bq.linear16(z(4, 8), far, out=far)
    far = z(1, 1, 8).expand(2 ** 31, 2, 8)
    with pytest.raises(ValueError):
        bq.attention(z(4, 2, 8), far, far)
    with pytest.raises(ValueError):
        bq.attention(far, z(4, 2, 8), z(4, 2, 8), out=far)


def test_references():
    x, w, g, r = z(4, 64), z(32, 64), z(2, 32), z(4, 32)
    q, lens = z(4, 2, 64), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    long = z(20000, 8, 64)

    def calls():
        bq.linear16(x, w, gate=g, residual=r)
        bq.linear16(x, w, out=r, workspace=ws)
        bq.layer_norm(x, scale=z(2, 64), shift=z(2, 64))
        bq.attention(q, q, q, cu_seqlens_q=lens, return_lse=True)
        bq.attention(long[:1], long, long)   # allocates a workspace
        for bad in (lambda: bq.linear16(x, w, out=g), lambda: bq.layer_norm(x, eps=-1.0),
                    lambda: bq.attention(q, q, q, scale=-1.0), lambda: bq.linear16(x, w, gate=g, group_rows=1)):
            with pytest.raises((ValueError, bq.SvdqError)):
                bad()

    calls()
    torch.cuda.synchronize()
    held = [x, w, g, r, q, lens, ws, long, BF, torch.float32, torch.uint8, 64, 20000]
    gc.collect()
    counts, memory = [sys.getrefcount(t) for t in held], torch.cuda.memory_allocated()
    for _ in range(300):
        calls()
    torch.cuda.synchronize()
    gc.collect()
    assert torch.cuda.memory_allocated() == memory
    assert max(abs(sys.getrefcount(t) - n) for t, n in zip(held, counts)) < 100
