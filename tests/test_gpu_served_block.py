"""The served block end to end: its operators together, for prompts and then
token by token, against the same formulas in float64 torch around the cache's
and the linears' codes."""

import importlib.util
import math
import os
import sys

import pytest
import torch

import bit_quantized_diffusion_amd as bq
from tests._reference8 import blocks

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def _example():
    spec = importlib.util.spec_from_file_location("served_block", os.path.join(ROOT, "examples", "served_block.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod
    spec.loader.exec_module(mod)
    return mod


def _weight(pair):
    wq, ws = pair
    n, k = wq.shape
    return wq.double() * ws.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def _coded(x):
    """x as its codes stand for it."""
    m, k = x.shape
    pad = torch.nn.functional.pad(x, (0, blocks(k) * 128 - k)).view(m, -1, 128)
    s = pad.abs().amax(2, keepdim=True).clamp(min=2.0 ** -100) / 448
    return ((pad / s).float().to(torch.float8_e4m3fn).double() * s).view(m, -1)[:, :k]


def _norm(h, w):
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * w.double()


def _plain(x, residual, block, serving, new):
    """The block in float64, its values rounded where the block's tensors are."""
    hq, hk, d = block.heads, block.kv_heads, block.head_dim
    h = x.double() + residual.double()
    qkv = (_coded(_norm(h, block.norm1)) @ _weight(block.qkv).T).to(BF).double().view(-1, hq + 2 * hk, d)
    out = []
    t0 = 0
    for b, n in enumerate(new):
        length = int(serving.lengths[b])
        keys, values = serving.cache.read(serving.table[b], length)          # what the block put there
        q = qkv[t0:t0 + n, :hq]
        row = serving.rope[length - n:length].double()
        c, s = row[:, None, :d // 2], row[:, None, d // 2:]
        q = torch.cat([q[..., :d // 2] * c - q[..., d // 2:] * s, q[..., d // 2:] * c + q[..., :d // 2] * s], -1).to(BF).double()
        keys, values = (v.double().repeat_interleave(hq // hk, 1).transpose(0, 1).contiguous() for v in (keys, values))
        scores = torch.bmm(q.transpose(0, 1).contiguous(), keys.transpose(1, 2).contiguous()) / math.sqrt(d)
        at = torch.arange(length, device=x.device)
        scores.masked_fill_(at[None, :] > (at[length - n:, None]), -math.inf)
        out.append(torch.bmm(torch.softmax(scores, -1), values).transpose(0, 1).reshape(n, hq * d))
        t0 += n
    y = (_coded(torch.cat(out).to(BF).double()) @ _weight(block.out).T).to(BF).double()
    h = h.to(BF).double() + y
    z = _coded(_norm(h, block.norm2)) @ _weight(block.up).T
    z = torch.nn.functional.gelu(z, approximate="tanh").to(BF).double()
    return _coded(z) @ _weight(block.down).T, h


# A value that is off by d before it is rounded to a code of step s moves the
# code with probability d / s, by s: its square by d s on average.  Steps are at
# most 2^-3 of a value, so a relative error e comes out of a rounding to codes,
# and of the linear behind it, as sqrt(e 2^-3) at most.  The roundings to bf16
# and of P differ by 2^-8 at most: attention's output enters the output
# projection's codes with that, and the stream behind it (H) carries
# sqrt(2^-8 2^-3); the MLP's two linears (Y) round to codes once each again.
H = (2.0 ** -8 * 2.0 ** -3) ** 0.5
Y = ((H * 2.0 ** -3) ** 0.5 * 2.0 ** -3) ** 0.5


def _close(got, want, bound):
    off = got.double() - want
    assert got.isfinite().all()
    # single values: five times their root mean square, where the largest result is about four times its own
    assert off.norm() <= bound * want.norm() and off.abs().max() <= 2 * bound * want.abs().max(), (float(off.norm() / want.norm()), float(off.abs().max()))


def test_prompts_then_tokens():
    ex = _example()
    block = ex.random_block(512, 8, 2)
    new = [150, 1, 63, 64, 200]
    serving = ex.Serving.start(block, 5, 300)
    cu = torch.tensor([sum(new[:i]) for i in range(6)], dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(2)
    x, r = (torch.randn(sum(new), 512, generator=gen).to(BF).cuda() for _ in range(2))
    serving.lengths += cu.diff()
    y, h = ex.run_block(x, r, block, serving, cu)
    want, want_h = _plain(x, r, block, serving, new)
    _close(h, want_h, H)
    _close(y, want, Y)
    # keys and values in the cache are the projection's
    h0 = x.double() + r.double()
    qkv = (_coded(_norm(h0, block.norm1)) @ _weight(block.qkv).T).view(-1, 12, 64)
    _, values = serving.cache.read(serving.table[4], 200)
    v = qkv[-200:, 10:]
    assert (values - v).norm() <= 0.05 * v.norm()
    # token by token, over a page's border, eagerly and from a graph
    last = (cu[1:] - 1).long()
    x, h = y[last].clone(), h[last].clone()
    for _ in range(2):
        serving.lengths += 1
        y, h1 = ex.run_block(x, h, block, serving)
        want, want_h = _plain(x, h, block, serving, [1] * 5)
        _close(h1, want_h, H)
        _close(y, want, Y)
        x, h = y, h1
    x, h = x.clone(), h.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y, h1 = ex.run_block(x, h, block, serving)
    for _ in range(3):
        serving.lengths += 1
        graph.replay()
        torch.cuda.synchronize()
        want, want_h = _plain(x, h, block, serving, [1] * 5)
        _close(h1, want_h, H)
        _close(y, want, Y)
        x.copy_(y)
        h.copy_(h1)


def test_a_prompt_in_chunks_and_at_once():
    """The same tokens in one call or in several: near each other, page by page."""
    ex = _example()
    block = ex.random_block(256, 4, 2, seed=3)
    x = torch.randn(192, 256, generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    zero = torch.zeros_like(x)

    def cu(*n):
        return torch.tensor([0, *n], dtype=torch.int32, device="cuda")

    one, two = ex.Serving.start(block, 1, 192), ex.Serving.start(block, 1, 192)
    one.lengths += 192
    whole, _ = ex.run_block(x, zero, block, one, cu(192))
    parts = []
    for i in range(0, 192, 64):
        two.lengths += 64
        parts.append(ex.run_block(x[i:i + 64], zero[i:i + 64], block, two, cu(64))[0])
    _close(torch.cat(parts), whole.double(), Y)
