"""Plain 64-bit references of the 8-bit operators and the error bounds that
follow from how the kernels round (CPU, torch float64).

Unit roundoffs as in _reference16; a rounding to e4m3 is off by at most 2^-4
of the value, or by 2^-10 below 2^-6 (half its step of 2^-9)."""

import torch

from tests._reference16 import TINY, U16, U32, _group_rows, linear16_reference  # noqa: F401

F8 = torch.float8_e4m3fn
U8, TINY8 = 2.0 ** -4, 2.0 ** -10


def blocks(n):
    return -(-n // 128)


def code_bound(value, error):
    """How far a code may be from the value it rounds, known up to `error`."""
    a = value.abs() + error
    return error + torch.maximum(a * U8, torch.full_like(a, TINY8))


def quantize_plain(x):
    """The rule of svdq.h in fp32, step by step: (codes, scales)."""
    x = x.detach().cpu().float()
    m, k = x.shape
    pad = torch.nn.functional.pad(x, (0, blocks(k) * 128 - k)).view(m, -1, 128)
    s = torch.nan_to_num(pad.abs(), nan=0.0, posinf=float("inf")).amax(2).clamp(min=2.0 ** -100) / 448.0
    codes = (pad * (1.0 / s)[:, :, None]).view(m, -1)[:, :k].to(F8)
    return codes, s.t().contiguous()


def pack_plain(w):
    w = w.detach().cpu().float()
    n, k = w.shape
    pad = torch.nn.functional.pad(w, (0, blocks(k) * 128 - k, 0, blocks(n) * 128 - n)).view(blocks(n), 128, blocks(k), 128)
    s = pad.abs().amax(3).amax(1).clamp(min=2.0 ** -100) / 448.0
    codes = (pad * (1.0 / s)[:, None, :, None]).view(blocks(n) * 128, -1)[:n, :k].to(F8)
    return codes, s


def rms_reference(x, residual, weight, eps):
    """(h, bound of h's rounding, y, bound of the fp32 y) in float64.

    h is one fp32 sum; the K squares' sum is off by at most (K + 2) u32 of
    itself and 2 u32 from each h; the root halves that and takes a few u32 with
    the reciprocal; two products follow."""
    dtype = x.dtype
    h = x.detach().cpu().double()
    K = h.shape[1]
    if residual is not None:
        h = h + residual.detach().cpu().double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.detach().cpu().double()
    rel = ((K + 4) / 2 + 1 + 1 + 8) * U32
    return h, h.abs() * (U16[dtype] + 2 * U32) + TINY[dtype], y, y.abs() * rel + 2.0 ** -140


def _cut(xq, wq):
    """Sum over the groups of 8 consecutive k of the unit below which the matrix
    core cuts their products, and of its square: [blocks of 128][m][n] each.

    Measured on gfx950 with one product of 2^E and one of 3.515625 = 11.100001b
    in a group: all of the latter comes back for E <= 6, 3.5 for E = 8 to 12,
    2.0 for 14 and nothing for 16, either sign, and all of it whenever the two
    lie in different groups.  So the unit is 2^(E - 13), E the largest sum of
    two factors' exponents in the group (those below 2^-6 have that of 2^-6)."""
    device = "cuda" if torch.cuda.is_available() else "cpu"
    x, w = (torch.frexp(t.to(device).float())[1].clamp(min=-5) - 1 for t in (xq, wq))
    x, w = (torch.nn.functional.pad(t, (0, blocks(t.shape[1]) * 128 - t.shape[1]), value=-6) for t in (x, w))
    x, w = (torch.exp2(t.float()) for t in (x, w))       # whole exponents
    total, square = [], []
    for g in range(0, x.shape[1], 128):
        t = torch.zeros(x.shape[0], w.shape[0], device=device)
        s = torch.zeros_like(t)
        for c in range(g, g + 128, 8):
            top = torch.zeros_like(t)
            for k in range(c, c + 8):
                top = torch.maximum(top, x[:, k, None] * w[None, :, k])
            unit = top * 2.0 ** -13
            t += unit
            s += unit * unit
        total.append(t.cpu())
        square.append(s.cpu())
    return torch.stack(total).double(), torch.stack(square).double()


def gemm_reference(xq, xs, wq, ws, bias, act, gate, residual, group_rows, dtype):
    """(y, bound, expected root mean square of the error) in float64.

    In a block the matrix core cuts up to 7 products of each group of 8 by less
    than their unit; that aside its sums, like the blocks', are fp32: 2 u32 a
    term (cut or rounded) for 128, u32 a block and two for the scales.  The
    cuts go towards zero, so for codes of either sign they are independent, of
    mean zero and at most unit^2 / 3 each in the square.  The epilogue is
    linear16's."""
    total, square = _cut(xq, wq)
    xq, xs, wq, ws = (t.detach().cpu().double() for t in (xq, xs, wq, ws))
    (m, k), n = xq.shape, wq.shape[0]
    scale_w = ws.repeat_interleave(128, 0)[:n]
    x = xq * xs.t().repeat_interleave(128, 1)[:, :k]
    w = wq * scale_w.repeat_interleave(128, 1)[:, :k]
    lost, spread = torch.zeros(m, n, dtype=torch.float64), torch.zeros(m, n, dtype=torch.float64)
    for g in range(blocks(k)):
        s = xs[g][:, None] * scale_w[:, g][None, :]
        lost += 7 * total[g] * s
        spread += 7 / 3 * square[g] * s * s
    mag = x.abs() @ w.abs().T
    dz = lost + (2 * 128 + blocks(k) + 5) * U32 * mag
    y, bound, slope = _epilogue(x @ w.T, mag, dz, bias, act, gate, residual, group_rows, dtype)
    mean_square = spread * slope ** 2 + ((U16[dtype] * y.abs()) ** 2 + TINY[dtype] ** 2) / 3
    return y, bound, float(mean_square.sum().sqrt())


def _epilogue(z, mag, dz, bias, act, gate, residual, group_rows, dtype):
    if bias is not None:
        z = z + bias.detach().cpu().double()
        dz = dz + 2 * U32 * (mag + bias.detach().cpu().double().abs())
    y, arg = z, torch.zeros_like(z)
    if act == "gelu":
        arg = 2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        y = z * torch.sigmoid(arg)
    elif act == "silu":
        arg, y = z, z * torch.sigmoid(z)
    slope = torch.full_like(z, 1.13 if act != "none" else 1.0)
    dy = slope * dz + (8 * U32 + 6 * U32 * arg.abs().clamp(max=100)) * y.abs() + 2.0 ** -126
    if gate is not None:
        g = _group_rows(gate, z.shape[0], group_rows)
        y, dy, slope = y * g, dy * g.abs() + 2 * U32 * (y * g).abs(), slope * g.abs()
    if residual is not None:
        r = residual.detach().cpu().double()
        y, dy = y + r, dy + 2 * U32 * (y.abs() + r.abs())
    return y, dy + U16[dtype] * (y.abs() + dy) + TINY[dtype], slope
