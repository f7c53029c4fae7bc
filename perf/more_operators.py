"""Cases for the 8-bit serving path of a transformer block: the root-mean-square
norm that adds the residual and writes 8-bit codes, the 8-bit linear with a
scale for each block of 128, the cache of keys and values held in 8 bits
(appending to it, with the position rotation) and the attention that reads it.

``run`` computes a case in its plain form (elementary torch operations in
32 bits, one rounding at the end) or, where ``own`` is true, through the
library's entry points.  ``exact`` computes it in 64 bits from the
definition, apart from both.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_F8 = torch.float8_e4m3fn
_MOST = 448.0          # largest e4m3 value
_BLOCK = 128           # values of a row that share a scale
_PAGE = 64             # tokens of a cache page
_LOW, _HIGH = -40, 40  # exponents that a page's scale can take


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, m, k, dtype, residual=False, fp8=False):
    return {"name": name, "op": "norm", "m": m, "k": k, "dtype": dtype, "residual": residual, "fp8": fp8}


def _linear(name, m, k, n, dtype, codes=False, bias=False, act="none", gate=False, residual=False):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "dtype": dtype, "codes": codes, "bias": bias, "act": act,
            "gate": gate, "residual": residual}


def _append(name, new, old, heads_q, heads_k, head_dim, rotary, dtype, interleaved=False):
    return {"name": name, "op": "append", "new": new, "old": old, "heads_q": heads_q, "heads_k": heads_k, "head_dim": head_dim,
            "rotary": rotary, "dtype": dtype, "interleaved": interleaved}


def _attention(name, new, old, heads_q, heads_k, head_dim, dtype, causal=True, lse=False):
    return {"name": name, "op": "attention", "new": new, "old": old, "heads_q": heads_q, "heads_k": heads_k,
            "head_dim": head_dim, "dtype": dtype, "causal": causal, "lse": lse}


def listed():
    many = ",".join(str(3000 + 37 * (i * 29 % 64)) for i in range(64))
    return [
        # the norm before a block's projections while one token is decoded: latency
        _norm("norm token", 1, 4096, "bf16", residual=True, fp8=True),
        # the same for the tokens of a long prompt
        _norm("norm prompt", 4608, 4096, "bf16", residual=True, fp8=True),
        # fused QKV projection of eight sequences' next tokens: bound by reading the weights
        _linear("linear tokens", 8, 4096, 6144, "bf16", codes=True),
        # a short prompt of odd length into a narrower model, from 16-bit activations
        _linear("linear context", 333, 4096, 1536, "f16", bias=True),
        # first layer of an MLP with its activation, on codes from the norm
        _linear("linear mlp", 4608, 4096, 12288, "bf16", codes=True, bias=True, act="gelu"),
        # second layer of the MLP from 16-bit activations, with the block's gate and residual
        _linear("linear output", 4608, 12288, 4096, "bf16", gate=True, residual=True),
        # the next token of each of 64 sequences enters its last page
        _append("append tokens", ",".join(["1"] * 64), many, 32, 8, 128, 128, "bf16"),
        # a pack of prompts enters fresh and half-filled pages, half of each head rotated
        _append("append prompts", "1024,77,2048,1,333,0,1500,512,13,700", "0,0,640,100,31,5,0,1000,63,64", 32, 8, 128, 64, "f16",
                interleaved=True),
        # one short sequence in a small model: latency
        _attention("attention short", "1", "299", 12, 12, 64, "f16"),
        # one new token for each of eight sequences of very different lengths, with the statistics for a later merge
        _attention("attention one token", "1,1,1,1,1,1,1,1", "16383,9000,4096,0,12344,776,15999,63", 32, 8, 128, "bf16", lse=True),
        # a full decoding batch
        _attention("attention batch", ",".join(["1"] * 64), many, 32, 8, 128, "bf16"),
        # chunks of long prompts on top of what is cached, beside two sequences that decode
        _attention("attention chunk", "2048,1,1000,1", "6000,5000,333,77", 32, 8, 128, "bf16"),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _draw_norm(rng):
    m = _log_uniform(rng, 1, 16384)
    fp8 = rng.random() < 0.6
    step = 16 if fp8 else rng.choice([1, 8])
    k = max(step, _log_uniform(rng, 32, 16384) // step * step)
    while m * k > 4608 * 4096:
        m = (m + 1) // 2
    return _norm("", m, k, rng.choice(["bf16", "f16"]), residual=rng.random() < 0.6, fp8=fp8)


def _draw_linear(rng):
    m = rng.choice([_log_uniform(rng, 1, 64), _log_uniform(rng, 1, 4608), _log_uniform(rng, 64, 4608)])
    k = rng.choice([128, 16]) * _log_uniform(rng, 1, 128)
    n = rng.choice([1, 64]) * _log_uniform(rng, 16, 256) + rng.choice([0, 0, 1, 40])
    while m * k * n > 0.8 * 4608 * 4096 * 12288:
        m = (m + 1) // 2
    return _linear("", m, k, n, rng.choice(["bf16", "f16"]), codes=rng.random() < 0.5, bias=rng.random() < 0.5,
                   act=rng.choice(["none", "none", "gelu", "silu"]), gate=rng.random() < 0.3, residual=rng.random() < 0.4)


def _draw_heads(rng):
    heads_k = rng.choice([1, 2, 3, 4, 8, 10, 16])
    group = rng.choice([1, 1, 2, 3, 4, 5, 8])
    return heads_k * group if heads_k * group <= 32 else heads_k, heads_k, rng.choice([64, 64, 128, 128, 128, 32, 80, 96])


def _draw_append(rng):
    heads_q, heads_k, d = _draw_heads(rng)
    batch = rng.choice([1, 2, 3, 8, 20, 64])
    one = rng.random() < 0.5
    new = [1 if one else _log_uniform(rng, 1, 2048) for _ in range(batch)]
    while sum(new) > 8192:
        new = [(n + 1) // 2 for n in new]
    old = [0 if rng.random() < 0.2 else _log_uniform(rng, 1, 2048) for _ in range(batch)]
    return _append("", ",".join(map(str, new)), ",".join(map(str, old)), heads_q, heads_k, d, rng.choice([d, d, d // 2]),
                   rng.choice(["bf16", "f16"]), interleaved=rng.random() < 0.4)


def _draw_attention(rng):
    heads_q, heads_k, d = _draw_heads(rng)
    batch = rng.choice([1, 1, 2, 5, 8, 16, 48])
    kind = rng.choice(["token", "token", "few", "chunk"])
    new = [{"token": 1, "few": rng.choice([1, 2, 4, 7]), "chunk": _log_uniform(rng, 1, 2048)}[kind] for _ in range(batch)]
    old = [0 if rng.random() < 0.1 else _log_uniform(rng, 1, 16384) for _ in range(batch)]
    while sum(n + o for n, o in zip(new, old)) * heads_k * d > 2e8:
        old = [(n + 1) // 2 for n in old]
    while sum(n * (n + o) for n, o in zip(new, old)) * heads_q > 0.8 * 2048 * 8048 * 32:
        new = [(n + 1) // 2 for n in new]
    return _attention("", ",".join(map(str, new)), ",".join(map(str, old)), heads_q, heads_k, d, rng.choice(["bf16", "f16"]),
                      causal=rng.random() < 0.8, lse=rng.random() < 0.3)


def draw(rng):
    case = rng.choice([_draw_norm, _draw_linear, _draw_append, _draw_attention])(rng)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lens(text):
    return [int(n) for n in text.split(",")]


def _blocks(n, size=_BLOCK):
    return (n + size - 1) // size


def _row_codes(x32):
    """Codes and scales [blocks][rows] of a matrix, a scale for each 128 values of a row."""
    m, k = x32.shape
    pad = torch.nn.functional.pad(x32, (0, _blocks(k) * _BLOCK - k)).view(m, -1, _BLOCK)
    scale = pad.abs().amax(dim=2).clamp(min=2.0 ** -100) / _MOST
    codes = (pad * (1.0 / scale)[:, :, None]).view(m, -1)[:, :k].to(_F8)
    return codes, scale.t().contiguous()


def _weight_codes(w32):
    """Codes and scales [row blocks][blocks] of a weight, a scale for each 128 x 128 values."""
    n, k = w32.shape
    pad = torch.nn.functional.pad(w32, (0, _blocks(k) * _BLOCK - k, 0, _blocks(n) * _BLOCK - n))
    pad = pad.view(_blocks(n), _BLOCK, _blocks(k), _BLOCK)
    scale = pad.abs().amax(dim=(1, 3)).clamp(min=2.0 ** -100) / _MOST
    codes = (pad * (1.0 / scale)[:, None, :, None]).view(_blocks(n) * _BLOCK, -1)[:n, :k].to(_F8)
    return codes, scale


def _rope(positions, rotary):
    """cos and sin [positions][2][rotary / 2] of the rotation's angles."""
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda") * std + mean

    def channels(k, large):
        # 0.5 % of the channels far larger than the rest
        return torch.where(torch.rand((k,), generator=gen, device="cuda") < 0.005, large, 1.0)

    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        return {"case": case, "x": normal(m, k).to(dtype), "weight": normal(k, std=0.1, mean=1.0).to(dtype),
                "residual": (normal(m, k, std=2.0) * channels(k, 30.0)).to(dtype) if case["residual"] else None}
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        x = normal(m, k) * channels(k, 10.0)
        st = {"case": case, "bias": normal(n, std=0.1).to(dtype) if case["bias"] else None,
              "gate": normal(n, std=0.5).to(dtype) if case["gate"] else None,
              "residual": normal(m, n).to(dtype) if case["residual"] else None}
        st["wq"], st["ws"] = _weight_codes(normal(n, k, std=k ** -0.5))
        if case["codes"]:
            st["xq"], st["xs"] = _row_codes(x)
        else:
            st["x"] = x.to(dtype)
        return st
    new, old = _lens(case["new"]), _lens(case["old"])
    batch, hq, hk, d = len(new), case["heads_q"], case["heads_k"], case["head_dim"]
    total = [a + b for a, b in zip(new, old)]
    used = [_blocks(n, _PAGE) for n in total]
    width, pages = max(used) + 1, sum(used) + 5
    # pages in no order; entries past a sequence's end name none
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    st = {"case": case, "table": table, "lengths": torch.tensor(total, dtype=torch.int32, device="cuda"),
          "cu": torch.tensor([sum(new[:i]) for i in range(batch + 1)], dtype=torch.int32, device="cuda")}
    # codes that use their range, at scales that differ from page to page
    st["k8"] = torch.empty((pages, hk, _PAGE, d), dtype=_F8, device="cuda")
    st["v8"] = torch.empty((pages, hk, 4, d, 16), dtype=_F8, device="cuda")
    for codes in (st["k8"], st["v8"]):
        flat = codes.view(-1)
        for i in range(0, flat.numel(), 1 << 26):
            part = flat[i:i + (1 << 26)]
            part.copy_(normal(part.numel(), std=100.0).clamp_(-_MOST, _MOST))
    st["exponents"] = torch.randint(-8, -5, (pages, hk, 2), generator=gen, device="cuda").to(torch.int8)
    tokens = sum(new)
    if case["op"] == "append":
        qkv = normal(tokens, (hq + 2 * hk) * d).to(dtype)   # the fused projection's output, read in place
        st["q"] = qkv[:, :hq * d].view(tokens, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hk) * d].view(tokens, hk, d)
        st["v"] = qkv[:, (hq + hk) * d:].view(tokens, hk, d)
        st["rope"] = _rope(max(total), case["rotary"])
    else:
        st["q"] = normal(tokens, hq, d).to(dtype)
    if own:
        import bit_quantized_diffusion_amd as bq
        st["cache"] = bq.KVCache(st["k8"], st["v8"], st["exponents"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return {"norm": _run_norm, "linear": _run_linear, "append": _run_append, "attention": _run_attention}[state["case"]["op"]](state)


def _run_norm(st):
    case, x, weight, residual = st["case"], st["x"], st["weight"], st["residual"]
    if own:
        import bit_quantized_diffusion_amd as bq
        norm = bq.rms_norm_fp8 if case["fp8"] else bq.rms_norm
        return norm(x, weight, residual=residual, eps=1e-6)
    h = x.float()
    if residual is not None:
        h = h + residual.float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + 1e-6) * weight.float()
    out = _row_codes(y) if case["fp8"] else (y.to(x.dtype),)
    if residual is not None:
        out = (*out, h.to(x.dtype))
    return out if len(out) > 1 else out[0]


def _run_linear(st):
    case, wq, ws, bias, gate, residual = st["case"], st["wq"], st["ws"], st["bias"], st["gate"], st["residual"]
    dtype = _DTYPES[case["dtype"]]
    if own:
        import bit_quantized_diffusion_amd as bq
        more = dict(activation=case["act"], gate=gate, residual=residual)
        if case["codes"]:
            return bq.gemm_fp8(st["xq"], st["xs"], wq, ws, bias, dtype=dtype, **more)
        return bq.linear_fp8(st["x"], wq, ws, bias, **more)
    xq, xs = (st["xq"], st["xs"]) if case["codes"] else _row_codes(st["x"].float())
    n, k = wq.shape
    x32 = xq.float() * xs.t().repeat_interleave(_BLOCK, dim=1)[:, :k]
    w32 = wq.float() * ws.repeat_interleave(_BLOCK, dim=0)[:n].repeat_interleave(_BLOCK, dim=1)[:, :k]
    y = x32 @ w32.t()
    if bias is not None:
        y = y + bias.float()
    if case["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    elif case["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    if gate is not None:
        y = y * gate.float()
    if residual is not None:
        y = y + residual.float()
    return y.to(dtype)


def _power(e):
    """2^e of whole e in 32 bits, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _at(codes, *index):
    """Rows of a tensor of codes (taken as bytes)."""
    return codes.view(torch.uint8)[index].view(_F8)


def _rotate(x32, cos, sin, interleaved):
    """The first 2 * cos.shape[1] values of every head rotated, in x32's type."""
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    a, b = (x32[..., 0:2 * half:2], x32[..., 1:2 * half:2]) if interleaved else (x32[..., :half], x32[..., half:2 * half])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
    return torch.cat([turned, x32[..., 2 * half:]], dim=-1)


def _places(st):
    """Of every new token: its position, page and place in the page."""
    cu, lengths = st["cu"].long(), st["lengths"].long()
    at = torch.arange(st["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], at, right=True)
    position = lengths[seq] - cu[seq + 1] + at
    return position, st["table"].long()[seq, position // _PAGE], position % _PAGE


def _run_append(st):
    case = st["case"]
    k8, v8, exponents = st["k8"], st["v8"], st["exponents"]
    if own:
        import bit_quantized_diffusion_amd as bq
        q = bq.cache_append(st["cache"], st["k"], st["v"], st["table"], st["lengths"], q=st["q"], rope=st["rope"],
                            cu_seqlens=st["cu"], interleaved=case["interleaved"])
        return q, k8, v8, exponents
    pages, hk, _, d = k8.shape
    position, page, place = _places(st)
    cos, sin = st["rope"][position].chunk(2, dim=1)
    q = _rotate(st["q"].float(), cos, sin, case["interleaved"]).to(st["q"].dtype)
    k, v = _rotate(st["k"].float(), cos, sin, case["interleaved"]), st["v"].float()
    # the first new place of every page (64: none)
    first = torch.full((pages,), _PAGE, dtype=torch.long, device=k.device).scatter_reduce_(0, page, place, "amin")
    touched = (first < _PAGE).nonzero()[:, 0]
    first = first[touched]
    before = torch.arange(_PAGE, device=k.device)[None, :] < first[:, None]      # kept tokens of the page
    for new, which in ((k, 0), (v, 1)):
        top = torch.zeros((pages, hk), device=k.device)
        top.scatter_reduce_(0, page[:, None].expand(-1, hk), new.abs().amax(dim=2), "amax")
        fraction, power = torch.frexp(top[touched])
        need = torch.where(fraction > 0.875, power - 8, power - 9)               # the least e with top <= 448 * 2^e
        need = torch.where(top[touched] > 0, need, _LOW).clamp(_LOW, _HIGH).to(torch.int8)
        was = torch.where((first > 0)[:, None], exponents[touched, :, which], _LOW).to(torch.int8)
        now = torch.maximum(was, need)
        exponents[touched, :, which] = now
        shrink = _power(was - now)[:, :, None, None]
        if which == 0:
            old = _at(k8, touched).float()
            k8.view(torch.uint8)[touched] = torch.where(before[:, None, :, None], old * shrink, old).to(_F8).view(torch.uint8)
        else:
            old = _at(v8, touched).float().view(-1, hk, 4, d, 4, 4)
            kept = before.view(-1, 1, 4, 4, 4).transpose(2, 3)[:, :, :, None]      # [page][1][place / 4 % 4][1][place / 16][place % 4]
            old = torch.where(kept, old * shrink[..., None, None], old).view(-1, hk, 4, d, 16)
            v8.view(torch.uint8)[touched] = old.to(_F8).view(torch.uint8)
        codes = (new * _power(-exponents[page, :, which])[:, :, None]).clamp(-_MOST, _MOST).to(_F8)
        if which == 0:
            k8.view(torch.uint8)[page, :, place] = codes.view(torch.uint8)
        else:
            v8.view(torch.uint8)[page, :, place // 4 % 4, :, place // 16 * 4 + place % 4] = codes.view(torch.uint8)
    return q, k8, v8, exponents


def _run_attention(st):
    case, q, lengths = st["case"], st["q"], st["lengths"]
    if own:
        import bit_quantized_diffusion_amd as bq
        return bq.attention_paged(q, st["cache"], st["table"], lengths, cu_seqlens_q=st["cu"], causal=case["causal"],
                                  return_lse=case["lse"])
    tokens, hq, d = q.shape
    hk = case["heads_k"]
    group = hq // hk
    o = torch.zeros((tokens, hq, d), device=q.device)
    lse = torch.full((tokens, hq), -math.inf, device=q.device)
    q0 = 0
    for b, (new, old) in enumerate(zip(_lens(case["new"]), _lens(case["old"]))):
        n = new + old
        ids = st["table"][b, :_blocks(n, _PAGE)].long()
        scale = _power(st["exponents"][ids])                                       # [pages][heads][2]
        k = (_at(st["k8"], ids).float() * scale[:, :, 0, None, None]).transpose(0, 1).reshape(hk, -1, d)[:, :n]
        v = _at(st["v8"], ids).float().view(-1, hk, 4, d, 4, 4) * scale[:, :, 1, None, None, None, None]
        v = v.permute(1, 0, 4, 2, 5, 3).reshape(hk, -1, d)[:, :n].contiguous()
        rows = q[q0:q0 + new].float().view(new, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * new, d)
        s = torch.bmm(rows, k.transpose(1, 2).contiguous()).mul_(d ** -0.5).view(hk, group, new, n)
        if case["causal"] and new > 1:
            at = torch.arange(n, device=q.device)
            s.masked_fill_(at[None, :] > at[old:, None], -math.inf)
        top = s.amax(dim=-1, keepdim=True)
        p = s.sub_(top).exp_()
        total = p.sum(dim=-1, keepdim=True)
        out = torch.bmm(p.view(hk, group * new, n), v).view(hk, group, new, d) / total
        o[q0:q0 + new] = out.permute(2, 0, 1, 3).reshape(new, hq, d)
        lse[q0:q0 + new] = (top + total.log()).view(hq, new).t()
        q0 += new
    return (o.to(q.dtype), lse) if case["lse"] else o.to(q.dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        m, k, r = case["m"], case["k"], case["residual"]
        out = m * k + 4 * m * _blocks(k) if case["fp8"] else 2 * m * k
        return {"bytes": 2 * m * k * (3 if r else 1) + out + 2 * k, "flops": 6 * m * k}
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        x = m * k + 4 * m * _blocks(k) if case["codes"] else 2 * m * k
        vectors = 2 * n * (case["bias"] + case["gate"])
        return {"bytes": x + n * k + 4 * _blocks(n) * _blocks(k) + 2 * m * n * (2 if case["residual"] else 1) + vectors,
                "flops": 2 * m * n * k}
    new, old = _lens(case["new"]), _lens(case["old"])
    hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
    if case["op"] == "append":
        return {"bytes": sum(new) * d * (4 * hq + 6 * hk) + 4 * sum(new) * case["rotary"], "flops": 6 * sum(new) * (hq + hk) * d}
    pairs = sum(n * o + (n * (n + 1) // 2 if case["causal"] else n * n) for n, o in zip(new, old))
    moved = sum(n + o for n, o in zip(new, old)) * hk * 2 * d + 4 * sum(new) * hq * d + (4 * sum(new) * hq if case["lse"] else 0)
    return {"bytes": moved, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_codes(x):
    """What the codes of a matrix round, and its scales."""
    m, k = x.shape
    codes, scales = torch.empty_like(x), torch.empty((_blocks(k), m), dtype=torch.float64, device=x.device)
    for g in range(_blocks(k)):
        part = x[:, g * _BLOCK:(g + 1) * _BLOCK]
        scales[g] = torch.clamp(part.abs().max(dim=1).values, min=2.0 ** -100) / _MOST
        codes[:, g * _BLOCK:(g + 1) * _BLOCK] = part / scales[g][:, None]
    return codes, scales


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double()
        if case["residual"]:
            h = h + st["residual"].double()
        y = h / torch.sqrt((h ** 2).mean(1, keepdim=True) + 1e-6) * st["weight"].double()
        out = list(_exact_codes(y)) if case["fp8"] else [y]
        if case["residual"]:
            out.append(h)
        return out if len(out) > 1 else out[0]
    if case["op"] == "linear":
        n, k = st["wq"].shape
        if case["codes"]:
            x, xs = st["xq"].double(), st["xs"].double()
        else:
            # the codes are part of the definition: rounded once, from the quotient in 64 bits
            x, xs = _exact_codes(st["x"].double())
            x = x.float().to(_F8).double()
        z = torch.zeros((case["m"], n), dtype=torch.float64, device=x.device)
        ws = st["ws"].double()[torch.arange(n, device=x.device) // _BLOCK]
        for g in range(_blocks(k)):
            cut = slice(g * _BLOCK, (g + 1) * _BLOCK)
            z += (x[:, cut] @ st["wq"][:, cut].double().T) * xs[g][:, None] * ws[:, g][None, :]
        if st["bias"] is not None:
            z += st["bias"].double()
        if case["act"] == "gelu":
            z = torch.nn.functional.gelu(z, approximate="tanh")
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        if st["gate"] is not None:
            z = z * st["gate"].double()
        return z if st["residual"] is None else z + st["residual"].double()
    new, old = _lens(case["new"]), _lens(case["old"])
    hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
    if case["op"] == "append":
        return _exact_append(case, st, new, old, hk, d)
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    place = torch.arange(_PAGE, device="cuda")
    q0 = 0
    for b in range(len(new)):
        n = new[b] + old[b]
        ids = st["table"][b, :_blocks(n, _PAGE)].long()
        hidden = torch.arange(n, device="cuda")[None, :] > torch.arange(old[b], n, device="cuda")[:, None]
        for h in range(hk):
            powers = 2.0 ** st["exponents"][ids, h].double()
            keys = (_at(st["k8"], ids, h).double() * powers[:, 0, None, None]).reshape(-1, d)[:n]
            codes = _at(st["v8"], ids, h).double()[:, place // 4 % 4, :, place // 16 * 4 + place % 4]      # [place][pages][d]
            values = (codes.transpose(0, 1) * powers[:, 1, None, None]).reshape(-1, d)[:n]
            for i in range(h * hq // hk, (h + 1) * hq // hk):
                scores = (st["q"][q0:q0 + new[b], i].double() @ keys.T) / math.sqrt(d)
                if case["causal"]:
                    scores[hidden] = -math.inf
                lse[q0:q0 + new[b], i] = torch.logsumexp(scores, dim=1)
                o[q0:q0 + new[b], i] = torch.softmax(scores, dim=1) @ values
        q0 += new[b]
    return (o, lse) if case["lse"] else o


def _exact_append(case, st, new, old, hk, d):
    table, half = st["table"].cpu(), case["rotary"] // 2
    rope = st["rope"].double()
    position = torch.cat([torch.arange(o, o + n, device="cuda") for n, o in zip(new, old)])

    def turned(x):
        out = x.double().clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            c, s = rope[position, i][:, None], rope[position, half + i][:, None]
            out[..., a] = x[..., a].double() * c - x[..., b].double() * s
            out[..., b] = x[..., b].double() * c + x[..., a].double() * s
        return out

    q, k, v = turned(st["q"]), turned(st["k"]), st["v"].double()
    k8, v8, exponents = st["k8"].double(), st["v8"].double(), st["exponents"].clone()
    place = torch.arange(_PAGE, device="cuda")
    t0 = 0
    for b in range(len(new)):
        done = 0
        while done < new[b]:
            first = (old[b] + done) % _PAGE
            count = min(_PAGE - first, new[b] - done)
            page = int(table[b, (old[b] + done) // _PAGE])
            rows = slice(t0 + done, t0 + done + count)
            v_page = v8[page][:, place // 4 % 4, :, place // 16 * 4 + place % 4].permute(1, 0, 2).clone()   # [heads][place][d]
            for which, (fresh, held) in enumerate(((k[rows], k8[page]), (v[rows], v_page))):
                top = fresh.abs().amax(dim=(0, 2))
                need = torch.ceil(torch.log2(top.clamp(min=1e-300) / _MOST)).clamp(_LOW, _HIGH)
                was = exponents[page, :, which].double() if first else torch.full_like(need, _LOW)
                now = torch.maximum(was, need)
                held[:, :first] *= (2.0 ** (was - now))[:, None, None]
                held[:, first:first + count] = (fresh / (2.0 ** now)[None, :, None]).clamp(-_MOST, _MOST).transpose(0, 1)
                exponents[page, :, which] = now.to(torch.int8)
            v8[page] = v_page.view(hk, 4, 4, 4, d).permute(0, 2, 4, 1, 3).reshape(hk, 4, d, 16)
            done += count
        t0 += new[b]
    return q, k8, v8, exponents
