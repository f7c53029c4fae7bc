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
