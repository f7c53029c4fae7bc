"""The example block end to end: its 16-bit operators against the same
formulas in float32 torch around the same quantized layers."""

import importlib.util
import math
import os
import sys

import pytest
import torch

import bit_quantized_diffusion_amd as bq

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("transformer_block", os.path.join(ROOT, "examples", "transformer_block.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod
    spec.loader.exec_module(mod)
    return mod


def _plain(ex, x, timestep, block, lengths):
    """The block with torch operators (float32, rounded where the block's
    tensors are) and the library's quantized layers."""
    w, bf = block.width, torch.bfloat16

    def lin(v, weight, act=None):
        y = v.float() @ weight.float().t()
        return y * torch.sigmoid(y) if act else y

    t = lin(ex.sinusoid(timestep), block.embed1, True).to(bf)
    t = lin(t, block.embed2, True).to(bf)
    m = lin(t, block.modulation).to(bf)[0].float().split(w)

    def norm(v, shift, scale):
        v = v.float()
        off = v - v.mean(1, keepdim=True)
        return (off / torch.sqrt((off * off).mean(1, keepdim=True) + 1e-6) * (1 + scale) + shift).to(bf)

    qkv = bq.linear(norm(x, m[0], m[1]), block.qkv).float().view(-1, 3, block.heads, w // block.heads)
    parts = []
    for part in qkv.split(lengths):
        q, k, v = (part[:, i].transpose(0, 1).contiguous() for i in range(3))
        s = torch.matmul(q, k.transpose(1, 2).contiguous()) / math.sqrt(q.shape[2])
        parts.append(torch.matmul(torch.softmax(s, -1), v).transpose(0, 1).reshape(part.shape[0], w))
    a = torch.cat(parts).to(bf)
    x = (x.float() + m[2] * lin(a, block.out)).to(bf)
    return (x.float() + m[5] * bq.mlp(norm(x, m[3], m[4]), block.fc1, block.fc2).float()).to(bf)


def test_block_matches_plain_formulas():
    ex = _example()
    block = ex.random_block(256, 4, rank=16)
    lengths = [300, 77, 129]
    cu = torch.tensor([0, 300, 377, 506], dtype=torch.int32, device="cuda")
    x = torch.randn(506, 256, device="cuda").to(torch.bfloat16)
    got = ex.run_block(x, 0.3, block, cu).float()
    want = _plain(ex, x, 0.3, block, lengths).float()
    # a last-bit difference of an activation can move a 4-bit code: the
    # layers' stated bound, 1e-2 of the largest output
    assert got.isfinite().all()
    assert (got - want).abs().max() <= 1e-2 * want.abs().max()
    # sequences are apart: another image beside it changes nothing in one
    y = ex.run_block(x[:300], 0.3, block, cu[:2])
    assert (y.float() - got[:300]).abs().max() <= 1e-2 * want.abs().max()
