"""Plain 64-bit references of the 16-bit block operators and the error
bounds that follow from how the kernels round (CPU, torch float64).

Unit roundoffs: u = 2^-8 (bf16) or 2^-11 (fp16) for one rounding to nearest
even, 2^-24 for fp32."""

import math

import torch

U16 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# spacing of the subnormals, halved: the absolute part of a rounding
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
U32 = 2.0 ** -24


def attention_reference(q, k, v, lens_q, lens_k, causal, scale):
    """(o, lse, bound_o, bound_lse) in float64 on the CPU.

    A score is an fp32 sum of D products: off by at most D u32 scale
    sum |q||k|, plus two roundings in the exponent's argument (their size is
    that of the score and of the reference it is measured from).  A weight
    carries that error, the exponential's (below 4 u32) and one rounding to
    16 bits, a sum over n keys at most n u32 more.  The output is rounded
    once."""
    q, k, v = (t.detach().cpu() for t in (q, k, v))
    dtype = q.dtype
    u, tiny = U16[dtype], TINY[dtype]
    q, k, v = q.double(), k.double(), v.double()
    tq, hq, d = q.shape
    hk = k.shape[1]
    o = torch.zeros(tq, hq, d, dtype=torch.float64)
    lse = torch.full((tq, hq), -math.inf, dtype=torch.float64)
    bo = torch.zeros_like(o)
    bl = torch.zeros_like(lse)
    q0 = k0 = 0
    for nq, nk in zip(lens_q, lens_k):
        for h in range(hq):
            if nq == 0 or nk == 0:
                continue
            qq, kk, vv = q[q0:q0 + nq, h], k[k0:k0 + nk, h * hk // hq], v[k0:k0 + nk, h * hk // hq]
            hidden = torch.zeros(nq, nk, dtype=torch.bool)
            if causal:
                hidden = torch.arange(nk)[None, :] > torch.arange(nq)[:, None] + (nk - nq)
            # what a row cannot see does not enter, whatever it holds
            seen = ~hidden.all(dim=0)
            kk = torch.where(seen[:, None], kk, 0.0)
            vv = torch.where(seen[:, None], vv, 0.0)
            s = (qq @ kk.T * scale).masked_fill(hidden, -math.inf)
            mag = (qq.abs() @ kk.abs().T * scale).masked_fill(hidden, 0.0)
            row = torch.logsumexp(s, dim=1)
            empty = hidden.all(dim=1)
            p = torch.exp(s - torch.where(empty, 0.0, row)[:, None])
            lse[q0:q0 + nq, h] = row
            o[q0:q0 + nq, h] = p @ vv
            ds = ((d + 2) * mag.amax(dim=1) + 4 * s.masked_fill(hidden, 0.0).abs().amax(dim=1) + 8) * U32
            spread = p @ vv.abs()
            top = (~hidden).double() @ vv.abs()
            bo[q0:q0 + nq, h] = (u * o[q0:q0 + nq, h].abs() + (u + 2 * ds + 2 * (nk + 8) * U32)[:, None] * spread * (1 + u)
                                 + tiny * top + tiny)
            bl[q0:q0 + nq, h] = torch.where(empty, 0.0, ds + (nk + 8) * U32 + 2 * U32 * row.abs())
        q0, k0 = q0 + nq, k0 + nk
    return o, lse, bo, bl


def assert_within(got, want, bound, what):
    got, want = got.detach().cpu().double(), want
    same_inf = torch.isinf(want) & (got == want)
    bad = ~((got - want).abs() <= bound) & ~same_inf
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: "
                             f"{float(got[i])} against {float(want[i])}, bound {float(bound[i])}")


def _group_rows(t, rows, group_rows):
    """Row-wise view of a per-group matrix or of one vector."""
    t = t.detach().cpu().double()
    return t.expand(rows, -1) if t.dim() == 1 else t[torch.arange(rows) // group_rows]


def linear16_reference(x, w, bias, act, gate, residual, group_rows):
    """(y, bound) in float64 on the CPU.

    The sum of K products is off by at most K u32 sum |x||w| plus the bias's
    rounding; both activations have slopes of at most 1.13 and are evaluated
    to a few u32 of their argument's exponent (the exponential's argument is
    rounded: |t| u32 relative); gate and residual add one rounding each, the
    output one of 16 bits."""
    dtype = x.dtype
    u, tiny = U16[dtype], TINY[dtype]
    x, w = x.detach().cpu().double(), w.detach().cpu().double()
    z = x @ w.T
    mag = x.abs() @ w.abs().T
    if bias is not None:
        z = z + bias.detach().cpu().double()
        mag = mag + bias.detach().cpu().double().abs()
    dz = (x.shape[1] + 2) * U32 * mag
    if act == "gelu":
        arg = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        y = z * torch.sigmoid(arg)
    elif act == "silu":
        arg = z
        y = z * torch.sigmoid(z)
    else:
        arg, y = torch.zeros_like(z), z
    # past |arg| = 100 the exponential's own size (e^-100) bounds what is left
    dy = (1.13 * dz if act != "none" else dz) + (8 * U32 + 6 * U32 * arg.abs().clamp(max=100)) * y.abs() + 2.0 ** -126
    if gate is not None:
        g = _group_rows(gate, x.shape[0], group_rows)
        y, dy = y * g, dy * g.abs() + 2 * U32 * (y * g).abs()
    if residual is not None:
        r = residual.detach().cpu().double()
        y, dy = y + r, dy + 2 * U32 * (y.abs() + r.abs())
    return y, dy + u * (y.abs() + dy) + tiny


def layer_norm_reference(x, weight, bias, scale, shift, group_rows, eps):
    """(y, bound) in float64 on the CPU.

    The mean is off by at most (log-tree or chunk) K u32 mean|x|; a deviation
    by that and its own rounding; rstd by the relative error of the
    variance's sum (K u32) and of what the deviations carry into it; each
    product and sum after it rounds once."""
    dtype = x.dtype
    u, tiny = U16[dtype], TINY[dtype]
    x = x.detach().cpu().double()
    M, K = x.shape
    mean = x.mean(1, keepdim=True)
    off = x - mean
    var = (off * off).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    d_mean = (K + 2) * U32 * x.abs().mean(1, keepdim=True)
    d_off = d_mean + 2 * U32 * (off.abs() + d_mean)
    # variance: 2 E|off| d_mean + d_mean^2 and the sum's own rounding
    d_var = 2 * off.abs().mean(1, keepdim=True) * d_mean + d_mean ** 2 + (K + 4) * U32 * (var + eps)
    rel = d_var / (2 * (var + eps)) + 6 * U32
    y = off * rstd
    dy = d_off * rstd * (1 + rel) + y.abs() * (rel + 2 * U32)
    for t, op in ((weight, "*"), (bias, "+"), (scale, "1*"), (shift, "+")):
        if t is None:
            continue
        t = _group_rows(t, M, group_rows)
        if op == "+":
            y = y + t
            dy = dy + 2 * U32 * (y.abs() + t.abs() + dy)
        else:
            t = t + 1 if op == "1*" else t
            dy = dy * t.abs() * (1 + 4 * U32) + 4 * U32 * (y * t).abs()
            y = y * t
    return y, dy + u * (y.abs() + dy) + tiny
