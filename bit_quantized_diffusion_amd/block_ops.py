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
_MOST = 2 ** 31 - 2 ** 16


@functools.lru_cache(maxsize=4096)
def _strides(*values):
    """The C array of these strides."""
    return (ctypes.c_int64 * len(values))(*values)


# The smallest calls take longer on the host than on the device, so a valid
# argument is passed by one cheap look; the words are found for one that is not.


def _operand(t, dims, name, layout):
    """(dtype code, device index) of a call's first operand."""
    try:
        code, device = _DTYPE.get(t.dtype), t.get_device()
        stride = t.stride()
        if code is not None and device >= 0 and len(stride) == dims and (stride[-1] == 1 or t.shape[-1] <= 1):
            return code, device
    except (AttributeError, RuntimeError):
        raise TypeError(f"{name}: expected a device tensor {layout}") from None
    if code is None:
        raise TypeError(f"{name}: expected a bfloat16 or float16 tensor, got {t.dtype}")
    if len(stride) == dims and device >= 0:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    raise TypeError(f"{name}: expected a device tensor {layout}")


def _like(t, dtype, device, shape, name):
    """`t` is a tensor of this dtype, device and shape with a dense last
    dimension."""
    try:
        if (t.dtype is dtype and t.get_device() == device and t.shape == shape
                and (t.stride(-1) == 1 or shape[-1] <= 1)):
            return
    except (AttributeError, RuntimeError):
        raise TypeError(f"{name}: expected a device tensor") from None
    if t.dtype is not dtype or t.get_device() != device:
        raise TypeError(f"{name}: expected {dtype} on cuda:{device}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: the last dimension must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(device, fn, *args):
    """Run a library call with `device` current, on its current stream."""
    if device == _current_device():
        status = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status:
        check(status)


# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _workspace(workspace, nbytes, device):
    """(pointer, bytes, tensor kept alive): "auto" allocates on the call's
    stream, None gives none, a uint8 tensor is used as it is."""
    if workspace is None:
        return None, 0, None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 device tensor")
        if not nbytes:
            return None, 0, None
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=torch.device("cuda", device))
    elif workspace.dtype != torch.uint8 or workspace.get_device() != device or not workspace.is_contiguous():
        raise TypeError("workspace: expected a contiguous uint8 tensor on the call's device")
    return workspace.data_ptr(), workspace.numel(), workspace


@functools.lru_cache(maxsize=4096)
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
    sequences' starts (0 first, the total last); without them the tokens form
    one sequence, and cu_seqlens_k defaults to cu_seqlens_q.  causal counts
    from the sequences' ends (query i sees keys j <= i + len_k - len_q).
    scale defaults to head_dim ** -0.5.

    Returns o (like q, contiguous unless `out` is given, which overlaps none
    of q, k and v) or, with
    return_lse, (o, lse fp32 [total_q][heads_q]).  A query that sees no key
    gives o = 0, lse = -inf."""
    code, device = _operand(q, 3, "q", "[tokens][heads][head_dim]")
    total_q, heads_q, head_dim = q.shape
    dtype = q.dtype
    try:
        shape = k.shape
        total_k, heads_k, _ = shape
    except (AttributeError, ValueError):
        raise TypeError("k: expected a device tensor [tokens][heads][head_dim]") from None
    _like(k, dtype, device, (total_k, heads_k, head_dim), "k")
    _like(v, dtype, device, shape, "v")
    if total_q > _MOST or total_k > _MOST:
        raise ValueError("attention: more tokens than the library counts (2^31 - 2^16)")
    batch = 1
    cu_q = cu_k = None
    if cu_seqlens_q is None:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k without cu_seqlens_q")
    else:
        batch = _cu_seqlens(cu_seqlens_q, device, "cu_seqlens_q")
        if cu_seqlens_k is None:
            if total_k != total_q:
                raise ValueError("cu_seqlens_k is needed where q and k have different numbers of tokens")
            cu_seqlens_k = cu_seqlens_q
        elif cu_seqlens_k is not cu_seqlens_q and _cu_seqlens(cu_seqlens_k, device, "cu_seqlens_k") != batch:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same number of entries")
        cu_q, cu_k = cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr()
    sq, sk, sv, so = q.stride(), k.stride(), v.stride(), (heads_q * head_dim, head_dim)
    if out is None:
        out = q.new_empty(total_q, heads_q, head_dim)
    else:
        _like(out, dtype, device, q.shape, "out")
        so = out.stride()
    lse = q.new_empty((total_q, heads_q), dtype=torch.float32) if return_lse else None
    if total_q > 1 and total_k > 1 and heads_q > 1 and heads_k > 1:
        strides = _strides(sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1])
    else:
        # dimensions of size 1 have no stride, and get that of a dense tensor
        st = []
        for (token, head, *_), n, h in ((sq, total_q, heads_q), (sk, total_k, heads_k), (sv, total_k, heads_k),
                                        (so, total_q, heads_q)):
            st += (token if n > 1 else h * head_dim, head if h > 1 else head_dim)
        strides = _strides(*st)
    nbytes = 0 if workspace is None else attention_workspace_size(total_q, total_k, batch, heads_q, heads_k, head_dim)
    ws, ws_bytes, _keep = _workspace(workspace, nbytes, device)
    _call(device, lib.svdq_attention, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(lse), cu_q, cu_k,
          batch, total_q, total_k, heads_q, heads_k, head_dim, strides,
          (head_dim or 1) ** -0.5 if scale is None else float(scale), 1 if causal else 0, code, ws, ws_bytes)
    return (out, lse) if return_lse else out


def _cu_seqlens(cu, device, name):
    """Number of sequences."""
    if cu.dtype is not torch.int32 or cu.get_device() != device or cu.dim() != 1 or not cu.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous int32 tensor [batch+1] on cuda:{device}")
    batch = cu.shape[0] - 1
    if batch < 1:
        raise ValueError(f"{name}: expected batch + 1 >= 2 entries")
    return batch


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


def _grouped(t, dtype, device, rows, width, group_rows, name):
    """A per-group matrix [groups][width] or one vector [width]: checked
    against the rows it has to cover.  Returns (pointer, row stride, groups,
    rows of a group)."""
    try:
        shape = t.shape
    except AttributeError:
        raise TypeError(f"{name}: expected a device tensor") from None
    if len(shape) == 1:
        _like(t, dtype, device, (width,), name)
        return t.data_ptr(), width, 1, max(rows, 1)
    _like(t, dtype, device, (shape[0], width) if len(shape) == 2 else (0, width), name)
    groups = shape[0]
    if group_rows is None:
        if not groups or rows % groups:
            raise ValueError(f"{name}: {rows} rows do not divide into {groups} groups; pass group_rows")
        group_rows = max(rows // groups, 1)
    if group_rows < 1 or -(-rows // group_rows) > groups:
        raise ValueError(f"{name}: {groups} groups of {group_rows} rows do not cover {rows} rows")
    return t.data_ptr(), t.stride(0) if groups > 1 else width, groups, group_rows


def linear16(x, w, bias=None, *, activation: str = "none", gate=None, residual=None, group_rows=None, out=None,
             workspace="auto"):
    """residual + gate * act(x w^T + bias) in 16 bits with fp32 arithmetic
    and one rounding.

    x [M][K], w [N][K] (nn.Linear layout), bias [N], residual [M][N]; gate
    [N], or [groups][N] with row r taking group r // group_rows (group_rows
    defaults to M / groups).  activation: "none", "gelu" (tanh form) or
    "silu".  Rows may be strided.  `out` may be `residual`."""
    code, device = _operand(x, 2, "x", "[M][K]")
    M, K = x.shape
    dtype = x.dtype
    try:
        N, _ = w.shape
    except (AttributeError, ValueError):
        raise TypeError("w: expected a device tensor [N][K]") from None
    _like(w, dtype, device, (N, K), "w")
    if M > _MOST or N > _MOST:
        raise ValueError("linear16: more rows than the library counts (2^31 - 2^16)")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation: expected one of {tuple(ACTIVATIONS)}, got {activation!r}")
    if bias is not None:
        _like(bias, dtype, device, (N,), "bias")
    gate_ptr, ld_gate, _, rows = (None, 0, 1, 1) if gate is None else \
        _grouped(gate, dtype, device, M, N, group_rows, "gate")
    if residual is not None:
        _like(residual, dtype, device, (M, N), "residual")
    if out is None:
        out = x.new_empty(M, N)
    else:
        _like(out, dtype, device, (M, N), "out")
    if M == 0:
        return out
    nbytes = 0 if workspace is None else linear16_workspace_size(M, N, K)
    ws, ws_bytes, _keep = _workspace(workspace, nbytes, device)
    _call(device, lib.svdq_linear16, x.data_ptr(), _ld(x), w.data_ptr(), _ld(w), _ptr(bias), gate_ptr, ld_gate, rows,
          _ptr(residual), 0 if residual is None else _ld(residual), out.data_ptr(), _ld(out), M, N, K, act, code, ws,
          ws_bytes)
    return out


def layer_norm(x, weight=None, bias=None, *, scale=None, shift=None, group_rows=None, eps: float = 1e-6, out=None):
    """Adaptive layer norm over the last dimension of x [M][K]:
    (x - mean) rstd [* weight + bias] [* (1 + scale) + shift], fp32 arithmetic,
    one rounding.

    weight, bias [K]; scale, shift [K], or [groups][K] with row r taking group
    r // group_rows (group_rows defaults to M / groups).  Rows may be
    strided.  `out` may be x."""
    code, device = _operand(x, 2, "x", "[M][K]")
    M, K = x.shape
    dtype = x.dtype
    if M > _MOST:
        raise ValueError("layer_norm: more rows than the library counts (2^31 - 2^16)")
    if weight is not None:
        _like(weight, dtype, device, (K,), "weight")
    if bias is not None:
        _like(bias, dtype, device, (K,), "bias")
    scale_ptr = shift_ptr = None
    rows, ld = 1, K
    if scale is not None:
        scale_ptr, ld, groups, rows = _grouped(scale, dtype, device, M, K, group_rows, "scale")
    if shift is not None:
        shift_ptr, ld_shift, shift_groups, shift_rows = _grouped(shift, dtype, device, M, K, group_rows, "shift")
        if scale is not None and (shift_rows != rows or shift_groups != groups or (ld_shift != ld and groups > 1)):
            raise ValueError("scale and shift must have the same groups and row stride")
        rows, ld = shift_rows, ld_shift
    if out is None:
        out = x.new_empty(M, K)
    else:
        _like(out, dtype, device, (M, K), "out")
    if M == 0:
        return out
    _call(device, lib.svdq_layer_norm, x.data_ptr(), _ld(x), _ptr(weight), _ptr(bias), scale_ptr, shift_ptr, ld, rows,
          out.data_ptr(), _ld(out), M, K, eps, code)
    return out
