"""Plain 64-bit references of the paged 8-bit cache and the attention that
reads it, and the error bounds that follow from how the kernels round (CPU,
torch float64)."""

import math

import torch

import bit_quantized_diffusion_amd as bq
from tests._reference16 import TINY, U16, U32
from tests._reference8 import F8, code_bound

PAGE = bq.PAGE


def random_cache(pages, heads, d, gen, low=-6, high=2):
    """Codes over their whole range, exponents that differ from page to page."""
    def codes(*shape):
        return (torch.randn(shape, generator=gen) * 100).clamp(-448, 448).to(F8).cuda()
    e = torch.randint(low, high + 1, (pages, heads, 2), generator=gen).to(torch.int8).cuda()
    return bq.KVCache(codes(pages, heads, PAGE, d), codes(pages, heads, 4, d, 16), e)


def tables(lengths, gen, spare=2, width=None, extra=3):
    """A block table with pages in no order, -1 past the sequences' ends; and the number of pages."""
    used = [-(-max(n, 0) // PAGE) for n in lengths]
    order = torch.randperm(sum(used) + extra, generator=gen)
    table = torch.full((len(lengths), width or max(used) + spare), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        n = min(n, table.shape[1])
        table[b, :n] = order[at:at + n].int()
        at += n
    return table.cuda(), sum(used) + extra


def starts(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def by_place(v):
    """Values' codes as [pages][heads][64][head_dim] (bytes)."""
    pages, heads, _, d, _ = v.shape
    return v.view(torch.uint8).view(pages, heads, 4, d, 4, 4).permute(0, 1, 4, 2, 5, 3).reshape(pages, heads, PAGE, d)


class Snapshot:
    """The cache before a call, on the CPU; codes as bytes, by place."""

    def __init__(self, cache):
        self.k, self.v = cache.k.view(torch.uint8).cpu().clone(), by_place(cache.v).cpu().clone()
        self.e = cache.exponents.cpu().clone()


def turned(x, positions, rope, interleaved):
    """(rotated, bound of the fp32 arithmetic) of [tokens][heads][d] in float64."""
    x = x.detach().cpu().double()
    if rope is None:
        return x, torch.zeros_like(x)
    rope = rope.cpu().double()
    half = rope.shape[1] // 2
    row = rope[positions.clamp(0, rope.shape[0] - 1)]
    c, s = row[:, None, :half], row[:, None, half:]
    y, bound = x.clone(), torch.zeros_like(x)
    ia = torch.arange(half) * 2 if interleaved else torch.arange(half)
    ib = ia + (1 if interleaved else half)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    # two products and a sum, each rounded
    bound[..., ia] = 2 * U32 * ((a * c).abs() + (b * s).abs())
    bound[..., ib] = 2 * U32 * ((b * c).abs() + (a * s).abs())
    return y, bound


def exponent_of(top):
    """The least e with top <= 448 * 2^e, cut to [-40, 40]."""
    if top == 0:
        return -40
    m, p = math.frexp(top)
    return min(40, max(-40, p - 8 if m > 0.875 else p - 9))


def check_append(before, cache, k, v, table, lengths, new, rope=None, interleaved=False, first=0):
    """Every byte of the cache after a call, against the state before it.
    `new`: tokens of each sequence, the first of them at token `first`."""
    table, lengths = table.cpu(), lengths.cpu()
    pages = before.e.shape[0]
    k8, v8, e = before.k.clone(), before.v.clone(), before.e.clone()
    got_k, got_v = cache.k.view(torch.uint8).cpu(), by_place(cache.v).cpu()
    t0 = first
    for b, n in enumerate(new):
        length = int(lengths[b])
        positions = torch.arange(length - n, length)
        for which, x in ((0, k), (1, v)):
            rows = x[t0:t0 + n]
            if which == 0:
                y, err = turned(rows, positions, rope, interleaved)
            else:
                y, err = rows.detach().cpu().double(), torch.zeros(rows.shape, dtype=torch.float64)
            for p in sorted({int(i) // PAGE for i in positions if 0 <= i < table.shape[1] * PAGE}):
                page = int(table[b, p])
                if not 0 <= page < pages:
                    continue
                at = [i for i, q in enumerate(positions.tolist()) if q // PAGE == p and q >= 0]
                place = positions[at[0]].item() % PAGE
                codes, got = (k8, got_k) if which == 0 else (v8, got_v)
                for h in range(y.shape[1]):
                    part, part_err = y[at, h], err[at, h]
                    finite = torch.where(part.isfinite(), part.abs(), 0.0)
                    was = min(40, max(-40, int(before.e[page, h, which]))) if place else -40
                    now = max(was, exponent_of(float(finite.max())))
                    e[page, h, which] = now
                    if now > was and place:
                        old = codes[page, h, :place].view(F8).float() * 2.0 ** (was - now)
                        codes[page, h, :place] = old.to(F8).view(torch.uint8)
                    value = (part * 2.0 ** -now).clamp(-448, 448)
                    seen = got[page, h, place:place + len(at)].view(F8).double()
                    assert torch.equal(seen.isnan(), ~part.isfinite()), (b, p, h, which)
                    off = (seen - value).abs()
                    bad = ~(off <= code_bound(value, part_err * 2.0 ** -now)) & part.isfinite()
                    assert not bad.any(), (b, p, h, which, float(off[bad].max()))
                    codes[page, h, place:place + len(at)] = got[page, h, place:place + len(at)]   # checked above
        t0 += n
    assert torch.equal(cache.exponents.cpu(), e)
    assert torch.equal(got_k, k8), "keys: a byte that the call does not own"
    assert torch.equal(got_v, v8), "values: a byte that the call does not own"


def paged_reference(q, cache, table, lengths, new, causal, scale, first=0):
    """(o, lse, bound_o, bound_lse) in float64.

    As attention_reference of _reference16; the exponent's argument carries the
    page's exponent (up to 40, with two roundings of it).  A weight is rounded
    to 16 bits beside the codes: below their subnormals it is off by `tiny` of
    the largest weight, 2^ev of whose page the other codes then count with."""
    dtype = q.dtype
    u, tiny = U16[dtype], TINY[dtype]
    qd, table, lengths = q.detach().cpu().double(), table.cpu(), lengths.cpu()
    k8, v8, e = cache.k.view(torch.uint8).cpu(), by_place(cache.v).cpu(), cache.exponents.cpu().double().clamp(-40, 40)
    tokens, hq, d = qd.shape
    hk = k8.shape[1]
    o = torch.zeros(tokens, hq, d, dtype=torch.float64)
    lse = torch.full((tokens, hq), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    t0 = first
    for b, n in enumerate(new):
        length = min(max(int(lengths[b]), 0), table.shape[1] * PAGE)
        at = torch.arange(length)
        page = table[b, at // PAGE].long()
        there = (page >= 0) & (page < k8.shape[0])
        page = torch.where(there, page, 0)
        hidden = torch.zeros(n, length, dtype=torch.bool) | ~there[None, :]
        if causal:
            hidden |= at[None, :] > torch.arange(n)[:, None] + (max(int(lengths[b]), 0) - n)
        for h in range(hq if length and n else 0):
            g = h * hk // hq
            power = torch.exp2(e[page, g])                                        # [keys][2]
            keys = torch.where(there[:, None], k8[page, g, at % PAGE].view(F8).double(), 0.0) * power[:, :1]
            codes = torch.where(there[:, None], v8[page, g, at % PAGE].view(F8).double(), 0.0)
            seen = ~hidden.all(dim=0)
            keys, codes = torch.where(seen[:, None], keys, 0.0), torch.where(seen[:, None], codes, 0.0)
            values = codes * power[:, 1:]
            rows = qd[t0:t0 + n, h]
            s = (rows @ keys.T * scale).masked_fill(hidden, -math.inf)
            mag = (rows.abs() @ keys.abs().T * scale).masked_fill(hidden, 0.0)
            row = torch.logsumexp(s, dim=1)
            empty = hidden.all(dim=1)
            p = torch.exp(s - torch.where(empty, 0.0, row)[:, None])
            lse[t0:t0 + n, h] = row
            o[t0:t0 + n, h] = p @ values
            ds = ((d + 2) * mag.amax(dim=1) + 4 * s.masked_fill(hidden, 0.0).abs().amax(dim=1) + 8 + 4 * 40) * U32
            spread = p @ values.abs()
            top = (~hidden).double() @ codes.abs() * power[seen, 1].amax() if seen.any() else 0.0
            bo[t0:t0 + n, h] = (u * o[t0:t0 + n, h].abs() + (u + 2 * ds + 2 * (length + 8) * U32)[:, None] * spread * (1 + u)
                                + tiny * top + tiny)
            bl[t0:t0 + n, h] = torch.where(empty, 0.0, ds + (length + 8) * U32 + 2 * U32 * row.abs())
        t0 += n
    # past the largest value and half a step (fp16: 65520) a rounding gives an
    # infinity: exponents to 2^40 take fp16's results there.  Where what the
    # bound allows lies on both sides, either may come
    most = torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4)
    bo = torch.where(o.abs() + bo > most, torch.where(o.abs() - bo > most, bo, math.inf), bo)
    o = torch.where(o.abs() - bo > most, torch.copysign(torch.full_like(o, math.inf), o), o)
    return o, lse, bo, bl
