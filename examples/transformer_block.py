"""One modulated transformer block as an image model runs it: the quantized
W4A4 projections and the 16-bit operators between them.

    python examples/transformer_block.py [--tokens 4608] [--width 3072] [--heads 24]

The timestep's embedding gives six vectors (shift, scale and gate of each
half); each half is norm -> projections -> gated residual:

    x = x + gate1 * out(attention(qkv(norm(x) (1 + scale1) + shift1)))
    x = x + gate2 * mlp(norm(x) (1 + scale2) + shift2)

The fused QKV projection and the MLP are packed W4A4 layers; the embedder,
the modulation and the output projection stay in 16 bits.  Several images are
packed one after another (`lengths`); tokens attend within their own.
"""

from __future__ import annotations

import argparse
import math
import os
import sys
from dataclasses import dataclass

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_quantized_diffusion_amd as bq  # noqa: E402

EMBED = 256   # width of the timestep's sinusoid


@dataclass
class Block:
    """Weights of one block, resident on the device."""
    width: int
    heads: int
    embed1: torch.Tensor       # [width][EMBED]
    embed2: torch.Tensor       # [width][width]
    modulation: torch.Tensor   # [6 width][width]
    out: torch.Tensor          # [width][width]
    qkv: bq.PackedLinear       # width -> 3 width
    fc1: bq.PackedLinear       # width -> 4 width
    fc2: bq.PackedLinear       # 4 width -> width


def random_block(width: int, heads: int, rank: int = 32, seed: int = 0, device="cuda") -> Block:
    """A block with random weights, packed on the CPU."""
    rng = np.random.default_rng(seed)

    def dense(n, k, std=None):
        w = rng.standard_normal((n, k), dtype=np.float32) * np.float32(k ** -0.5 if std is None else std)
        return torch.from_numpy(w).to(torch.bfloat16)

    def packed(n, k):
        bits = dense(n, k).view(torch.int16).numpy().view(np.uint16)
        host = bq.pack_weights(bits, np.full(k, 4.0, np.float32), rank)
        return bq.PackedLinear.from_host(host, None, rank, device=device)

    return Block(width=width, heads=heads, embed1=dense(width, EMBED).to(device), embed2=dense(width, width).to(device),
                 modulation=dense(6 * width, width, 0.3 * width ** -0.5).to(device), out=dense(width, width).to(device),
                 qkv=packed(3 * width, width), fc1=packed(4 * width, width), fc2=packed(width, 4 * width))


def sinusoid(timestep: float, device="cuda") -> torch.Tensor:
    half = EMBED // 2
    freq = torch.exp(-math.log(10000.0) * torch.arange(half, device=device, dtype=torch.float32) / half)
    arg = 1000.0 * timestep * freq
    return torch.cat([arg.cos(), arg.sin()])[None].to(torch.bfloat16)


def run_block(x: torch.Tensor, timestep: float, block: Block, cu_seqlens: torch.Tensor) -> torch.Tensor:
    """x bf16 [tokens][width] -> the block's output, the same shape."""
    w, tokens = block.width, x.shape[0]
    t = bq.linear16(sinusoid(timestep, x.device), block.embed1, activation="silu")
    t = bq.linear16(t, block.embed2, activation="silu")
    shift1, scale1, gate1, shift2, scale2, gate2 = bq.linear16(t, block.modulation)[0].split(w)

    h = bq.layer_norm(x, scale=scale1, shift=shift1)
    qkv = bq.linear(h, block.qkv).view(tokens, 3, block.heads, w // block.heads)
    a = bq.attention(qkv[:, 0], qkv[:, 1], qkv[:, 2], cu_seqlens_q=cu_seqlens)   # read in place
    x = bq.linear16(a.view(tokens, w), block.out, gate=gate1, residual=x)

    h = bq.layer_norm(x, scale=scale2, shift=shift2)
    return torch.addcmul(x, gate2, bq.mlp(h, block.fc1, block.fc2))


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1024, help="tokens of the first of two images; the second has a third fewer")
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--heads", type=int, default=8)
    args = ap.parse_args()
    block = random_block(args.width, args.heads)
    lengths = [args.tokens, args.tokens - args.tokens // 3]
    cu = torch.tensor([0, lengths[0], sum(lengths)], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lengths), args.width, device="cuda").to(torch.bfloat16)
    for timestep in (1.0, 0.5, 0.1):
        x = run_block(x, timestep, block, cu)
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(10):
        run_block(x, 0.5, block, cu)
    end.record()
    end.synchronize()
    print(f"{sum(lengths)} tokens, width {args.width}, {args.heads} heads: {begin.elapsed_time(end) / 10:.3f} ms a block, "
          f"output std {x.float().std().item():.3f}")


if __name__ == "__main__":
    main()
