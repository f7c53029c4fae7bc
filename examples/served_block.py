"""A text model's decoder block served in 8 bits: the 8-bit linears between the
norms that write their codes, and attention over the paged 8-bit cache.

    python examples/served_block.py [--batch 8] [--prompt 1024] [--width 2048] [--heads 16] [--kv-heads 4]

    h = x + residual;  q, k, v = split(Wqkv norm(h));  rotate q and k, k and v into the cache
    x = Wout attention(q, cache);  h = x + h;  x = Wdown gelu(Wup norm(h))

Prompts of different lengths enter together, then every sequence goes on by one
token a step; the same calls serve both.
"""

from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_quantized_diffusion_amd as bq  # noqa: E402


@dataclass
class Block:
    """Weights of one block, resident on the device: (codes, scales) of each linear."""
    heads: int
    kv_heads: int
    head_dim: int
    norm1: torch.Tensor
    norm2: torch.Tensor
    qkv: tuple
    out: tuple
    up: tuple
    down: tuple


def random_block(width: int, heads: int, kv_heads: int, seed: int = 0, device="cuda") -> Block:
    """A block with random weights, packed on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    d = width // heads

    def packed(n, k):
        wq, ws = bq.pack_fp8((torch.randn(n, k, generator=gen) * k ** -0.5).to(torch.bfloat16))
        return wq.to(device), ws.to(device)

    def weight():
        return (1 + 0.1 * torch.randn(width, generator=gen)).to(torch.bfloat16).to(device)

    return Block(heads, kv_heads, d, weight(), weight(), packed((heads + 2 * kv_heads) * d, width), packed(width, width),
                 packed(4 * width, width), packed(width, 4 * width))


@dataclass
class Serving:
    """The sequences' cache and where they stand in it."""
    cache: bq.KVCache
    table: torch.Tensor      # [batch][pages of the longest sequence]
    lengths: torch.Tensor    # tokens in the cache
    rope: torch.Tensor

    @classmethod
    def start(cls, block: Block, batch: int, most: int, device="cuda") -> "Serving":
        width = -(-most // bq.PAGE)
        order = torch.randperm(batch * width, generator=torch.Generator().manual_seed(1)).int()   # pages in any order
        return cls(bq.KVCache.allocate(batch * width, block.kv_heads, block.head_dim, device), order.view(batch, width).to(device),
                   torch.zeros(batch, dtype=torch.int32, device=device), bq.rope_table(most, block.head_dim, device=device))


def run_block(x, residual, block: Block, serving: Serving, cu_seqlens=None):
    """New tokens x bf16 [tokens][width] (one a sequence, or packed at
    `cu_seqlens`) and the residual stream before them -> the same two after the
    block.  `serving.lengths` counts them already."""
    hq, hk, d = block.heads, block.kv_heads, block.head_dim
    tokens = x.shape[0]
    codes, scales, h = bq.rms_norm_fp8(x, block.norm1, residual=residual)
    qkv = bq.gemm_fp8(codes, scales, *block.qkv).view(tokens, hq + 2 * hk, d)
    q, k, v = qkv.split([hq, hk, hk], dim=1)                                    # read in place
    q = bq.cache_append(serving.cache, k, v, serving.table, serving.lengths, q=q, rope=serving.rope, cu_seqlens=cu_seqlens)
    a = bq.attention_paged(q, serving.cache, serving.table, serving.lengths, cu_seqlens_q=cu_seqlens)
    x = bq.linear_fp8(a.view(tokens, hq * d), *block.out)
    codes, scales, h = bq.rms_norm_fp8(x, block.norm2, residual=h)
    return bq.linear_fp8(bq.gemm_fp8(codes, scales, *block.up, activation="gelu"), *block.down), h


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1024, help="tokens of the first prompt; each of the others has a tenth fewer")
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=4)
    args = ap.parse_args()
    block = random_block(args.width, args.heads, args.kv_heads)
    lens = [max(1, int(args.prompt * 0.9 ** i)) for i in range(args.batch)]
    serving = Serving.start(block, args.batch, args.prompt + 64)
    cu = torch.tensor([sum(lens[:i]) for i in range(args.batch + 1)], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), args.width, device="cuda").to(torch.bfloat16)
    serving.lengths += cu.diff()
    y, h = run_block(x, torch.zeros_like(x), block, serving, cu)
    last = (cu[1:] - 1).long()
    x, h = y[last], h[last]
    torch.cuda.synchronize()
    # a step's launches in a graph; lengths and inputs change under it
    step_x, step_h = x.clone(), h.clone()
    serving.lengths += 1
    run_block(step_x, step_h, block, serving)   # before capture, as any kernel's first call
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out_x, out_h = run_block(step_x, step_h, block, serving)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        graph.replay()
        serving.lengths += 1
    end.record()
    end.synchronize()
    print(f"{args.batch} sequences of {min(lens)} to {max(lens)} tokens, width {args.width}, {args.heads}/{args.kv_heads} heads: "
          f"{begin.elapsed_time(end) / 20 * 1000:.0f} us a step, output std {out_x.float().std().item():.3f}")


if __name__ == "__main__":
    main()
