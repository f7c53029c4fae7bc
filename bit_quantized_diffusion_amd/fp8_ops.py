"""The 8-bit operators of a transformer block that is served in 8 bits: thin
bindings over the C ABI (``include/svdq.h``), with torch tensors for device
memory and streams.  Codes are torch.float8_e4m3fn.

Forward only: results carry no gradient.  The arguments are checked by the
extension ``_block_ops``, as those of the 16-bit operators are.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from ._lib import BF16, F16, check, lib
from .block_ops import ACTIVATIONS, _block_ops

FP8_BLOCK = 128     # values along K that share a scale
PAGE = 64           # tokens of a page of the cache


def pack_fp8(w):
    """Codes and scales of a weight, on the CPU: w [N][K] bf16 or fp16 host
    tensor -> (wq [N][K] float8_e4m3fn, ws fp32 [ceil(N / 128)][ceil(K / 128)]),
    a scale for each 128 x 128 values.  K % 16 == 0."""
    if not isinstance(w, torch.Tensor) or w.device.type != "cpu" or w.dtype not in (torch.bfloat16, torch.float16) or w.dim() != 2:
        raise TypeError("w: expected a bfloat16 or float16 host tensor [N][K]")
    w = w.detach().contiguous()
    n, k = w.shape
    wq = torch.empty((n, k), dtype=torch.uint8)
    ws = torch.empty((-(-n // FP8_BLOCK), -(-k // FP8_BLOCK)), dtype=torch.float32)
    check(lib.svdq_pack_fp8(w.data_ptr(), k, n, BF16 if w.dtype == torch.bfloat16 else F16, wq.data_ptr(), ws.data_ptr()))
    return wq.view(torch.float8_e4m3fn), ws


def quantize_fp8(x):
    """Codes and scales of activations x [M][K] (bf16 or fp16, rows may be
    strided, K % 16 == 0): (xq [M][K] float8_e4m3fn, xs fp32
    [ceil(K / 128)][M]), a scale for each 128 values of a row."""
    return _block_ops.quantize_fp8(x)


def rms_norm_fp8(x, weight=None, *, residual=None, eps: float = 1e-6, residual_out=None):
    """`rms_norm` with its result in codes: (yq, ys), or with a residual
    (yq, ys, h), yq and ys as from `quantize_fp8` but taken from the fp32
    result (one rounding).  K % 16 == 0."""
    return _block_ops.rms_norm(x, weight, residual, eps, None, residual_out, True)


def _activation(name: str) -> int:
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation: expected one of {tuple(ACTIVATIONS)}, got {name!r}")
    return act


def gemm_fp8(xq, xs, wq, ws, bias=None, *, dtype=torch.bfloat16, activation: str = "none", gate=None, residual=None,
             group_rows=None, out=None):
    """residual + gate * act(x w^T + bias) from codes and scales of x
    (`quantize_fp8`, `rms_norm_fp8`) and w (`pack_fp8`), in `dtype` (bfloat16
    or float16; bias, gate, residual and `out` have it too).  Epilogue,
    `group_rows` and `out` as for `linear16`.  No gradient."""
    return _block_ops.gemm_fp8(xq, xs, wq, ws, bias, _activation(activation), gate, residual, group_rows, dtype, out)


def linear_fp8(x, wq, ws, bias=None, *, activation: str = "none", gate=None, residual=None, group_rows=None, out=None):
    """`gemm_fp8` of 16-bit activations x [M][K], whose codes are made on the
    way (`quantize_fp8`); the result has x's dtype."""
    return _block_ops.gemm_fp8(x, None, wq, ws, bias, _activation(activation), gate, residual, group_rows, None, out)


@dataclass
class KVCache:
    """Keys and values of many sequences in pages of 64 tokens, as 8-bit codes
    with an exponent for each page and head (value = code * 2^e).  The tensors
    are the user's, contiguous, on one device."""
    k: torch.Tensor            # float8_e4m3fn [pages][heads][64][head_dim]
    v: torch.Tensor            # float8_e4m3fn [pages][heads][4][head_dim][16]: place p at [p // 4 % 4][d][p // 16 * 4 + p % 4]
    exponents: torch.Tensor    # int8 [pages][heads][2], of keys and of values

    @classmethod
    def allocate(cls, pages: int, heads: int, head_dim: int, device="cuda") -> "KVCache":
        """An empty cache; what pages hold before tokens enter them is of no
        account, and starts as zeros."""
        codes = torch.zeros((2, pages * heads * PAGE * head_dim), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        return cls(codes[0].view(pages, heads, PAGE, head_dim), codes[1].view(pages, heads, 4, head_dim, 16),
                   torch.zeros((pages, heads, 2), dtype=torch.int8, device=device))

    def read(self, block_table_row, length: int):
        """(keys, values) of one sequence as fp32 [length][heads][head_dim], in
        plain torch operations: for inspection and tests.  As the attention
        sees them: exponents are cut to [-40, 40], and positions whose entry
        names no page, or past the row's end, hold zeros."""
        pages, heads, _, d = self.k.shape
        length = int(length)
        row = block_table_row.to(device=self.k.device, dtype=torch.long)
        ids = torch.full((-(-length // PAGE),), -1, dtype=torch.long, device=self.k.device)
        ids[:row.numel()] = row[:ids.numel()]
        there = (ids >= 0) & (ids < pages)
        ids = torch.where(there, ids, 0)
        scale = torch.exp2(self.exponents[ids].clamp(-40, 40).double()).float()
        k = self.k.view(torch.uint8)[ids].view(self.k.dtype).float() * scale[:, :, 0, None, None]
        v = self.v.view(torch.uint8)[ids].view(self.v.dtype).float() * scale[:, :, 1, None, None, None]
        v = v.view(ids.numel(), heads, 4, d, 4, 4).permute(0, 1, 4, 2, 5, 3).reshape(k.shape)
        k, v = (torch.where(there[:, None, None, None], t, 0.0).transpose(1, 2).reshape(ids.numel() * PAGE, heads, d)[:length]
                for t in (k, v))
        return k, v


def rope_table(positions: int, rotary: int, base: float = 10000.0, device="cuda"):
    """Angles of the position rotation for `cache_append`: fp32
    [positions][rotary], rotary / 2 cosines and as many sines of
    position * base ** (-2 i / rotary), taken in 64 bits."""
    freq = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().to(device)


def cache_append(cache: KVCache, k, v, block_table, lengths, *, q=None, rope=None, cu_seqlens=None, interleaved: bool = False,
                 q_out=None):
    """New tokens' keys and values into the cache, with the rotation by
    position on the way; returns the rotated q (or None without q).

    k, v [tokens][heads_k][head_dim], q [tokens][heads_q][head_dim], bf16 or
    fp16, any token and head strides (views into a fused QKV projection are
    read in place).  block_table int32 [batch][width]: the page of each 64
    positions (entries that name no page have none).  lengths int32 [batch]:
    tokens of each sequence, the new ones included; a sequence's new tokens are
    the last of its positions.  cu_seqlens int32 [batch + 1]: the sequences'
    starts in the pack; without it each has one token.  rope: from
    `rope_table`, its width is the number of values rotated of each head (a
    multiple of 16); pairs are i and i + rotary / 2, or 2 i and 2 i + 1 if
    `interleaved`.  `q_out` may be q.

    A page's exponent grows as its tokens ask for it, and its codes are then
    rescaled.  No gradient."""
    return _block_ops.cache_append(cache.k, cache.v, cache.exponents, block_table, lengths, cu_seqlens, k, v, q, rope, interleaved,
                                   q_out)


def attention_paged_workspace_size(total: int, batch: int, table_width: int, heads_q: int, heads_k: int, head_dim: int) -> int:
    """Bytes of workspace with which `attention_paged` cuts the keys of few
    queries into equal shares (0: it runs them in one piece anyway)."""
    out = ctypes.c_size_t(0)
    check(lib.svdq_attention_paged_workspace_size(total, batch, table_width, heads_q, heads_k, head_dim, ctypes.byref(out)))
    return int(out.value)


def attention_paged(q, cache: KVCache, block_table, lengths, *, cu_seqlens_q=None, causal: bool = True, scale=None, out=None,
                    return_lse: bool = False, workspace="auto"):
    """softmax(scale q k^T) v over sequences in the cache.

    q [tokens][heads_q][head_dim], bf16 or fp16, strides multiples of 8;
    heads_q is a multiple of the cache's heads, and query head h reads key
    head h // (heads_q // heads_k).  block_table, lengths and cu_seqlens_q
    as for `cache_append`, which runs before: q's tokens are the last of
    their sequences.  causal: query i of n sees keys j <= i + length - n.  scale
    defaults to head_dim ** -0.5.  workspace: as for `attention`.

    Returns o (like q, contiguous unless `out` is given, which overlaps no
    operand) or, with return_lse, (o, lse fp32 [tokens][heads_q]).  A query
    that sees no key gives o = 0, lse = -inf.  No gradient."""
    return _block_ops.attention_paged(cache.k, cache.v, cache.exponents, block_table, lengths, cu_seqlens_q, q, causal, scale, out,
                                      return_lse, workspace)
