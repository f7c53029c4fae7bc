"""The 16-bit operators of a transformer block that stand between its
quantized linears: thin bindings over the C ABI (``include/svdq.h``), with
torch tensors for device memory and streams.  bf16 and fp16.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import BF16, F16, check, lib

_DTYPE = {torch.bfloat16: BF16, torch.float16: F16}


def _dtype_code(t, name):
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected a bfloat16 or float16 tensor, got {t.dtype}")
    return code


def _like(t, ref, shape, name):
    """`t` is a device tensor of ref's device and dtype, of this shape and
    with a dense last dimension."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    if t.dtype != ref.dtype or t.device != ref.device:
        raise TypeError(f"{name}: expected {ref.dtype} on {ref.device}, got {t.dtype} on {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(device, fn, *args):
    """Run a library call with `device` current, on its current stream."""
    if device.index is not None and device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return check(fn(*args, torch.cuda.current_stream(device).cuda_stream))
    check(fn(*args, torch.cuda.current_stream(device).cuda_stream))


def _workspace(workspace, nbytes, device):
    """(pointer, bytes, tensor kept alive): "auto" allocates on the call's
    stream, None gives none, a uint8 tensor is used as it is."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 device tensor")
        if not nbytes:
            return None, 0, None
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=device)
    if workspace is None:
        return None, 0, None
    if workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise TypeError("workspace: expected a contiguous uint8 tensor on the call's device")
    return workspace.data_ptr(), workspace.numel(), workspace


@functools.lru_cache(maxsize=4096)
def attention_workspace_size(total_q: int, total_k: int, batch: int, heads_q: int, heads_k: int, head_dim: int) -> int:
    """Bytes of workspace with which `attention` cuts long key ranges into
    parts (0: it runs them in one piece anyway)."""
    out = ctypes.c_size_t(0)
    check(lib.svdq_attention_workspace_size(total_q, total_k, batch, heads_q, heads_k, head_dim, ctypes.byref(out)))
    return int(out.value)


def _strides(t):
    """Token and head strides; dimensions of size 1 have none, and get those
    of a dense tensor."""
    n, heads, d = t.shape
    return (t.stride(0) if n > 1 else heads * d), (t.stride(1) if heads > 1 else d)


def attention(q, k, v, *, cu_seqlens_q=None, cu_seqlens_k=None, causal: bool = False, scale=None, out=None,
              return_lse: bool = False, workspace="auto"):
    """softmax(scale q k^T) v over packed sequences.

    q [total_q][heads_q][head_dim], k and v [total_k][heads_k][head_dim],
    bf16 or fp16, with any token and head strides that are multiples of 8
    (views into a fused QKV projection are read in place).  heads_q is a
    multiple of heads_k; query head h reads key head h // (heads_q // heads_k).
    cu_seqlens_q, cu_seqlens_k: int32 device tensors [batch+1] with the
    sequences' starts (0 first, the total last); without them the tokens form
    one sequence, and cu_seqlens_k defaults to cu_seqlens_q.  causal counts
    from the sequences' ends (query i sees keys j <= i + len_k - len_q).
    scale defaults to head_dim ** -0.5.

    Returns o (like q, contiguous unless `out` is given) or, with
    return_lse, (o, lse fp32 [total_q][heads_q]).  A query that sees no key
    gives o = 0, lse = -inf."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise TypeError("q: expected a device tensor [tokens][heads][head_dim]")
    dtype = _dtype_code(q, "q")
    total_q, heads_q, head_dim = q.shape
    _like(q, q, None, "q")
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("k: expected a device tensor [tokens][heads][head_dim]")
    total_k, heads_k, _ = k.shape
    _like(k, q, (total_k, heads_k, head_dim), "k")
    _like(v, q, (total_k, heads_k, head_dim), "v")
    batch = 1
    if cu_seqlens_q is None:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k without cu_seqlens_q")
    else:
        if cu_seqlens_k is None:
            if total_k != total_q:
                raise ValueError("cu_seqlens_k is needed where q and k have different numbers of tokens")
            cu_seqlens_k = cu_seqlens_q
        for name, cu in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
            if cu.dtype != torch.int32 or cu.device != q.device or cu.dim() != 1 or not cu.is_contiguous():
                raise TypeError(f"{name}: expected a contiguous int32 tensor [batch+1] on {q.device}")
        batch = cu_seqlens_q.shape[0] - 1
        if batch < 1 or cu_seqlens_k.shape[0] != batch + 1:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must both have batch + 1 >= 2 entries")
    if out is None:
        out = torch.empty((total_q, heads_q, head_dim), dtype=q.dtype, device=q.device)
    else:
        _like(out, q, q.shape, "out")
    lse = torch.empty((total_q, heads_q), dtype=torch.float32, device=q.device) if return_lse else None
    strides = (ctypes.c_int64 * 8)(*_strides(q), *_strides(k), *_strides(v), *_strides(out))
    nbytes = attention_workspace_size(total_q, total_k, batch, heads_q, heads_k, head_dim) \
        if isinstance(workspace, str) else 0
    ws, ws_bytes, _keep = _workspace(workspace, nbytes, q.device)
    _call(q.device, lib.svdq_attention, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens_q),
          _ptr(cu_seqlens_k), batch, total_q, total_k, heads_q, heads_k, head_dim, strides,
          head_dim ** -0.5 if scale is None else float(scale), int(bool(causal)), dtype, ws, ws_bytes)
    return (out, lse) if return_lse else out


ACTIVATIONS = {"none": 0, "gelu": 1, "silu": 2}


@functools.lru_cache(maxsize=4096)
def linear16_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace with which `linear16` cuts small grids along K (0:
    it runs them in one piece anyway)."""
    out = ctypes.c_size_t(0)
    check(lib.svdq_linear16_workspace_size(M, N, K, ctypes.byref(out)))
    return int(out.value)


def _ld(t):
    """Row stride of a matrix (a single row has none, and gets its length)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _grouped(t, ref, rows, width, group_rows, name):
    """A per-group matrix [groups][width] or one vector [width]: checked
    against the rows it has to cover."""
    if isinstance(t, torch.Tensor) and t.dim() == 1:
        t = t.unsqueeze(0)
        group_rows = max(rows, 1)
    _like(t, ref, None, name)
    if t.dim() != 2 or t.shape[1] != width:
        raise ValueError(f"{name}: expected [groups][{width}] or [{width}], got {tuple(t.shape)}")
    if group_rows is None:
        if rows % t.shape[0]:
            raise ValueError(f"{name}: {rows} rows do not divide into {t.shape[0]} groups; pass group_rows")
        group_rows = rows // t.shape[0]
    if group_rows < 1 or -(-rows // group_rows) > t.shape[0]:
        raise ValueError(f"{name}: {t.shape[0]} groups of {group_rows} rows do not cover {rows} rows")
    return t, group_rows


def linear16(x, w, bias=None, *, activation: str = "none", gate=None, residual=None, group_rows=None, out=None,
             workspace="auto"):
    """residual + gate * act(x w^T + bias) in 16 bits with fp32 arithmetic
    and one rounding.

    x [M][K], w [N][K] (nn.Linear layout), bias [N], residual [M][N]; gate
    [N], or [groups][N] with row r taking group r // group_rows (group_rows
    defaults to M / groups).  activation: "none", "gelu" (tanh form) or
    "silu".  Rows may be strided.  `out` may be `residual`."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise TypeError("x: expected a device tensor [M][K]")
    dtype = _dtype_code(x, "x")
    _like(x, x, None, "x")
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise TypeError("w: expected a device tensor [N][K]")
    M, K = x.shape
    N = w.shape[0]
    _like(w, x, (N, K), "w")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation: expected one of {tuple(ACTIVATIONS)}, got {activation!r}")
    if bias is not None:
        _like(bias, x, (N,), "bias")
    rows = 1
    if gate is not None:
        gate, rows = _grouped(gate, x, M, N, group_rows, "gate")
    if residual is not None:
        _like(residual, x, (M, N), "residual")
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    else:
        _like(out, x, (M, N), "out")
    if M == 0:
        return out
    nbytes = linear16_workspace_size(M, N, K) if isinstance(workspace, str) else 0
    ws, ws_bytes, _keep = _workspace(workspace, nbytes, x.device)
    _call(x.device, lib.svdq_linear16, _ptr(x), _ld(x), _ptr(w), _ld(w), _ptr(bias), _ptr(gate),
          0 if gate is None else _ld(gate), rows, _ptr(residual), 0 if residual is None else _ld(residual), _ptr(out),
          _ld(out), M, N, K, act, dtype, ws, ws_bytes)
    return out


def layer_norm(x, weight=None, bias=None, *, scale=None, shift=None, group_rows=None, eps: float = 1e-6, out=None):
    """Adaptive layer norm over the last dimension of x [M][K]:
    (x - mean) rstd [* weight + bias] [* (1 + scale) + shift], fp32 arithmetic,
    one rounding.

    weight, bias [K]; scale, shift [K], or [groups][K] with row r taking group
    r // group_rows (group_rows defaults to M / groups).  Rows may be
    strided.  `out` may be x."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise TypeError("x: expected a device tensor [M][K]")
    dtype = _dtype_code(x, "x")
    _like(x, x, None, "x")
    M, K = x.shape
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _like(t, x, (K,), name)
    rows, ld = 1, 0
    if scale is not None:
        scale, rows = _grouped(scale, x, M, K, group_rows, "scale")
        ld = _ld(scale)
    if shift is not None:
        shift, shift_rows = _grouped(shift, x, M, K, group_rows, "shift")
        if scale is not None and (shift_rows != rows or (_ld(shift) != ld and scale.shape[0] > 1)):
            raise ValueError("scale and shift must have the same groups and row stride")
        rows, ld = shift_rows, max(ld, _ld(shift))
    if out is None:
        out = torch.empty((M, K), dtype=x.dtype, device=x.device)
    else:
        _like(out, x, (M, K), "out")
    if M == 0:
        return out
    _call(x.device, lib.svdq_layer_norm, _ptr(x), _ld(x), _ptr(weight), _ptr(bias), _ptr(scale), _ptr(shift), ld, rows,
          _ptr(out), _ld(out), M, K, float(eps), dtype)
    return out
