"""The 16-bit operators of a transformer block that stand between its
quantized linears: thin bindings over the C ABI (``include/svdq.h``), with
torch tensors for device memory and streams.  bf16 and fp16.

The arguments are checked, and the outputs allocated, by the extension
``_block_ops`` (``csrc/svdq_python.cpp``): the smallest calls take longer on the
host than on the device.  Without it these operators raise ImportError; the rest
of the package needs libsvdq.so alone.

Forward only: results carry no gradient, also where an operand requires one (the
quantized layers around them have none).
"""

from __future__ import annotations

import ctypes

import torch

from ._lib import check, lib   # loads torch's HIP runtime and libsvdq.so first


class _Missing:
    """In the place of an extension that is not there for this Python."""

    def __init__(self, why: ImportError):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{name} needs the extension _block_ops, built for this Python by "
                          f"`python bit_quantized_diffusion_amd/build.py`: {self._why}") from self._why


try:
    from . import _block_ops
except ImportError as e:
    _block_ops = _Missing(e)
else:
    # the current stream's handle without a Stream object around it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _block_ops.setup(torch.Tensor, torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int32, _raw_stream,
                     _current_device, torch.cuda.set_device, check, torch.float8_e4m3fn, torch.int8)


def attention_workspace_size(total_q: int, total_k: int, batch: int, heads_q: int, heads_k: int, head_dim: int) -> int:
    """Bytes of workspace with which `attention` cuts long key ranges into
    parts (0: it runs them in one piece anyway)."""
    out = ctypes.c_size_t(0)
    check(lib.svdq_attention_workspace_size(total_q, total_k, batch, heads_q, heads_k, head_dim, ctypes.byref(out)))
    return int(out.value)


def attention(q, k, v, *, cu_seqlens_q=None, cu_seqlens_k=None, causal: bool = False, scale=None, out=None,
              return_lse: bool = False, workspace="auto"):
    """softmax(scale q k^T) v over packed sequences.

    q [total_q][heads_q][head_dim], k and v [total_k][heads_k][head_dim],
    bf16 or fp16, with any token and head strides that are multiples of 8
    (views into a fused QKV projection are read in place).  heads_q is a
    multiple of heads_k; query head h reads key head h // (heads_q // heads_k).
    cu_seqlens_q, cu_seqlens_k: int32 device tensors [batch+1] with the
    sequences' starts (0 first, the total last; queries before the first or
    past the last are padding, and give o = 0, lse = -inf); without them the
    tokens form one sequence, and cu_seqlens_k defaults to cu_seqlens_q.  causal counts
    from the sequences' ends (query i sees keys j <= i + len_k - len_q).
    scale defaults to head_dim ** -0.5.  A NaN or infinity in v at a key that
    causal alone hides from a query can reach it.  workspace: "auto" allocates what the
    schedule takes, None gives none, a uint8 tensor is used as it is.

    Returns o (like q, contiguous unless `out` is given, which overlaps none
    of q, k and v) or, with return_lse, (o, lse fp32 [total_q][heads_q]).  A
    query that sees no key gives o = 0, lse = -inf.  No gradient."""
    return _block_ops.attention(q, k, v, cu_seqlens_q, cu_seqlens_k, causal, scale, out, return_lse, workspace)


ACTIVATIONS = {"none": 0, "gelu": 1, "silu": 2}


def linear16_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace with which `linear16` cuts small grids along K,
    whatever its operands' alignment (0: it runs them in one piece anyway)."""
    out = ctypes.c_size_t(0)
    check(lib.svdq_linear16_workspace_size(M, N, K, ctypes.byref(out)))
    return int(out.value)


def linear16(x, w, bias=None, *, activation: str = "none", gate=None, residual=None, group_rows=None, out=None,
             workspace="auto"):
    """residual + gate * act(x w^T + bias) in 16 bits with fp32 arithmetic
    and one rounding.

    x [M][K], w [N][K] (nn.Linear layout), bias [N], residual [M][N]; gate
    [N], or [groups][N] with row r taking group r // group_rows (group_rows
    defaults to M / groups).  activation: "none", "gelu" (tanh form) or
    "silu".  Rows may be strided.  `out` may be `residual`.  workspace: as
    for `attention`.  No gradient."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation: expected one of {tuple(ACTIVATIONS)}, got {activation!r}")
    return _block_ops.linear16(x, w, bias, act, gate, residual, group_rows, out, workspace)


def layer_norm(x, weight=None, bias=None, *, scale=None, shift=None, group_rows=None, eps: float = 1e-6, out=None):
    """Adaptive layer norm over the last dimension of x [M][K]:
    (x - mean) rstd [* weight + bias] [* (1 + scale) + shift], fp32 arithmetic,
    one rounding.

    weight, bias [K]; scale, shift [K], or [groups][K] with row r taking group
    r // group_rows (group_rows defaults to M / groups).  Rows may be
    strided.  `out` may be x.  No gradient."""
    return _block_ops.layer_norm(x, weight, bias, scale, shift, group_rows, eps, out)


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, out=None, residual_out=None):
    """Root-mean-square norm over the last dimension of h = x [+ residual]:
    h / sqrt(mean(h^2) + eps) [* weight], fp32 arithmetic, one rounding.

    x and residual [M][K], weight [K].  Rows may be strided.  Returns y, or
    with a residual (y, h): h is the sum, rounded once (y is taken from the
    unrounded one).  `out` may be x or residual, and so may `residual_out`;
    the two share no memory (ValueError).  No gradient."""
    return _block_ops.rms_norm(x, weight, residual, eps, out, residual_out, False)
