"""The 8-bit operators of a transformer block that is served in 8 bits: thin
bindings over the C ABI (``include/svdq.h``), with torch tensors for device
memory and streams.  Codes are torch.float8_e4m3fn.

Forward only: results carry no gradient.  The arguments are checked by the
extension ``_block_ops``, as those of the 16-bit operators are.
"""

from __future__ import annotations

import ctypes

import torch

from ._lib import BF16, F16, check, lib
from .block_ops import ACTIVATIONS, _block_ops

FP8_BLOCK = 128     # values along K that share a scale


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


def gemm_fp8_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace with which `gemm_fp8` cuts small grids along K (0: it
    runs them in one piece anyway)."""
    out = ctypes.c_size_t(0)
    check(lib.svdq_gemm_fp8_workspace_size(M, N, K, ctypes.byref(out)))
    return int(out.value)


def _activation(name: str) -> int:
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation: expected one of {tuple(ACTIVATIONS)}, got {name!r}")
    return act


def gemm_fp8(xq, xs, wq, ws, bias=None, *, dtype=torch.bfloat16, activation: str = "none", gate=None, residual=None,
             group_rows=None, out=None, workspace="auto"):
    """residual + gate * act(x w^T + bias) from codes and scales of x
    (`quantize_fp8`, `rms_norm_fp8`) and w (`pack_fp8`), in `dtype` (bfloat16
    or float16; bias, gate, residual and `out` have it too).  Epilogue,
    `group_rows`, `out` and workspace as for `linear16`.  No gradient."""
    return _block_ops.gemm_fp8(xq, xs, wq, ws, bias, _activation(activation), gate, residual, group_rows, dtype, out, workspace)


def linear_fp8(x, wq, ws, bias=None, *, activation: str = "none", gate=None, residual=None, group_rows=None, out=None,
               workspace="auto"):
    """`gemm_fp8` of 16-bit activations x [M][K], whose codes are made on the
    way (`quantize_fp8`); the result has x's dtype."""
    return _block_ops.gemm_fp8(x, None, wq, ws, bias, _activation(activation), gate, residual, group_rows, None, out, workspace)
