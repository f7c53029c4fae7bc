"""Cases for the operators around the quantized linears of a transformer
block: attention, the 16-bit linear with its epilogue, and the adaptive layer
norm.

``run`` computes a case in its plain form (elementary torch operations in
32 bits, one rounding at the end) or, where ``own`` is true, through the
library's entry points.  ``exact`` computes it in 64 bits from the
definition, apart from both.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attention(name, lens_q, lens_k, heads_q, heads_k, head_dim, dtype, causal=False, fused=False, lse=False):
    return {"name": name, "op": "attention", "lens_q": lens_q, "lens_k": lens_k, "heads_q": heads_q, "heads_k": heads_k,
            "head_dim": head_dim, "dtype": dtype, "causal": causal, "fused": fused, "lse": lse}


def _linear(name, m, k, n, dtype, act="none", gate=False, residual=False, groups=1):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "dtype": dtype, "act": act, "gate": gate,
            "residual": residual, "groups": groups}


def _norm(name, m, k, dtype, affine=False, modulate=True, groups=1):
    return {"name": name, "op": "norm", "m": m, "k": k, "dtype": dtype, "affine": affine, "modulate": modulate,
            "groups": groups}


def listed():
    return [
        # joint attention of a 1024x1024 image (4096 tokens) and its 512 text tokens, read from the fused QKV output
        _attention("attention joint", "4608", "4608", 24, 24, 128, "bf16", fused=True),
        # a pack of prompts of different lengths (one of them empty) through a causal text model with grouped heads
        _attention("attention prompts", "1024,77,2048,1,333,0,1500,512,13,700", "1024,77,2048,1,333,0,1500,512,13,700",
                   32, 8, 128, "bf16", causal=True, fused=True),
        # one short prompt through a small causal text encoder: latency
        _attention("attention encoder", "77", "77", 12, 12, 64, "f16", causal=True, fused=True),
        # two images' tokens reading their text tokens (cross attention), lengths of their own on each side
        _attention("attention cross", "4096,4096", "77,154", 10, 10, 64, "f16"),
        # one new token for each of eight sequences of very different lengths, with the statistics a later merge needs
        _attention("attention one token", "1,1,1,1,1,1,1,1", "16384,9001,4097,1,12345,777,16000,0", 32, 8, 128, "bf16",
                   causal=True, lse=True),
        # first layer of the timestep embedder for one image: latency
        _linear("linear embedder", 1, 256, 3072, "bf16", act="silu"),
        # modulation of a block (six vectors) for two images: bound by reading the weights
        _linear("linear modulation", 2, 3072, 18432, "bf16"),
        # text tokens into the model's width, an odd number of them
        _linear("linear context", 333, 4096, 3072, "f16"),
        # attention's output projection with the block's gate and residual
        _linear("linear output", 4608, 3072, 3072, "bf16", gate=True, residual=True),
        # first layer of an unquantized MLP with its activation
        _linear("linear mlp", 4608, 3072, 12288, "bf16", act="gelu"),
        # the norm before each projection of a block, modulated by the timestep
        _norm("norm block", 4608, 3072, "bf16"),
        # a text encoder's norm of one token with its own weight and bias: latency
        _norm("norm token", 1, 768, "f16", affine=True, modulate=False),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _draw_attention(rng):
    head_dim = rng.choice([64, 64, 128, 128, 128, 40, 80, 96])
    heads_k = rng.choice([1, 2, 3, 4, 8, 10, 16, 24])
    group = rng.choice([1, 1, 1, 2, 3, 4, 8])
    if heads_k * group > 32:
        group = 1
    batch = rng.choice([1, 1, 2, 3, 5, 8, 12])
    kind = rng.choice(["self", "self", "cross", "token"])
    lens_k = [0 if rng.random() < 0.05 else _log_uniform(rng, 1, 16384 if kind == "token" else 4608) for _ in range(batch)]
    if kind == "self":
        lens_q = list(lens_k)
    elif kind == "cross":
        lens_q = [_log_uniform(rng, 1, 4608) for _ in range(batch)]
    else:
        lens_q = [rng.choice([1, 1, 1, 2, 5]) for _ in range(batch)]
    # at most the work of the largest listed case, counted as the plain form does it (every query against every key of the pack)
    heads_q = heads_k * group
    while sum(lens_q) * sum(lens_k) * heads_q > 0.8 * 4608 * 4608 * 24:
        lens_q = [(n + 1) // 2 for n in lens_q]
        lens_k = list(lens_q) if kind == "self" else [(n + 1) // 2 for n in lens_k]
    if not sum(lens_k):
        lens_k[0] = 1
    if not sum(lens_q):
        lens_q[0] = 1
    causal = rng.random() < 0.5
    return _attention("", ",".join(map(str, lens_q)), ",".join(map(str, lens_k)), heads_q, heads_k, head_dim,
                      rng.choice(["bf16", "f16"]), causal=causal, fused=lens_q == lens_k and rng.random() < 0.5,
                      lse=rng.random() < 0.3)


def _odd(rng, value, step=8):
    """About half of the sizes stay as drawn, the others become multiples of `step`."""
    return value if rng.random() < 0.5 else max(step, value // step * step)


def _draw_linear(rng):
    m = rng.choice([_log_uniform(rng, 1, 16), _log_uniform(rng, 1, 4608), _log_uniform(rng, 64, 4608)])
    k = _odd(rng, _log_uniform(rng, 64, 15360))
    n = _odd(rng, _log_uniform(rng, 16, 18432))
    while m * k * n > 0.8 * 4608 * 3072 * 12288:
        k, n = max(64, k // 2), max(16, n // 2)
    groups = rng.choice([g for g in (1, 2, 3, 4) if m % g == 0])
    return _linear("", m, k, n, rng.choice(["bf16", "f16"]), act=rng.choice(["none", "none", "gelu", "silu"]),
                   gate=rng.random() < 0.3, residual=rng.random() < 0.4, groups=groups)


def _draw_norm(rng):
    m = _log_uniform(rng, 1, 16384)
    k = _odd(rng, _log_uniform(rng, 32, 12288))
    while m * k > 4608 * 12288:
        m = (m + 1) // 2
    groups = rng.choice([g for g in (1, 2, 3, 4) if m % g == 0])
    affine = rng.random() < 0.5
    return _norm("", m, k, rng.choice(["bf16", "f16"]), affine=affine, modulate=not affine or rng.random() < 0.5, groups=groups)


def draw(rng):
    case = rng.choice([_draw_attention, _draw_linear, _draw_norm])(rng)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lens(text):
    return [int(n) for n in text.split(",")]


def _cu_seqlens(lens):
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)

    if case["op"] == "attention":
        lens_q, lens_k = _lens(case["lens_q"]), _lens(case["lens_k"])
        tq, tk, hq, hk, d = sum(lens_q), sum(lens_k), case["heads_q"], case["heads_k"], case["head_dim"]
        if case["fused"]:
            # the fused projection's output [tokens][(Hq + 2 Hk) D], read in place
            qkv = normal(tq, (hq + 2 * hk) * d)
            q = qkv[:, :hq * d].view(tq, hq, d)
            k = qkv[:, hq * d:(hq + hk) * d].view(tk, hk, d)
            v = qkv[:, (hq + hk) * d:].view(tk, hk, d)
        else:
            q, k, v = normal(tq, hq, d), normal(tk, hk, d), normal(tk, hk, d)
        return {"case": case, "q": q, "k": k, "v": v, "cu_q": _cu_seqlens(lens_q), "cu_k": _cu_seqlens(lens_k)}
    m, k = case["m"], case["k"]
    group_rows = m // case["groups"]
    if case["op"] == "linear":
        n = case["n"]
        # activations with 0.5 % of the channels far larger than the rest, weights of about 1/sqrt(k)
        x = torch.randn((m, k), generator=gen, device="cuda")
        x *= torch.where(torch.rand((k,), generator=gen, device="cuda") < 0.005, 10.0, 1.0)
        return {"case": case, "x": x.to(dtype), "w": normal(n, k, std=k ** -0.5), "bias": normal(n, std=0.1),
                "gate": normal(case["groups"], n, std=0.5) if case["gate"] else None,
                "residual": normal(m, n) if case["residual"] else None, "group_rows": group_rows}
    # a residual stream: rows off centre, a few channels far larger than the rest
    x = torch.randn((m, k), generator=gen, device="cuda") + torch.randn((m, 1), generator=gen, device="cuda")
    x *= torch.where(torch.rand((k,), generator=gen, device="cuda") < 0.005, 30.0, 1.0)
    return {"case": case, "x": x.to(dtype), "weight": normal(k, std=0.1, mean=1.0) if case["affine"] else None,
            "bias": normal(k, std=0.1) if case["affine"] else None,
            "scale": normal(case["groups"], k, std=0.3) if case["modulate"] else None,
            "shift": normal(case["groups"], k, std=0.3) if case["modulate"] else None, "group_rows": group_rows}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return {"attention": _run_attention, "linear": _run_linear, "norm": _run_norm}[state["case"]["op"]](state)


def _run_attention(st):
    case, q, k, v = st["case"], st["q"], st["k"], st["v"]
    if own:
        import bit_quantized_diffusion_amd as bq
        return bq.attention(q, k, v, cu_seqlens_q=st["cu_q"], cu_seqlens_k=st["cu_k"], causal=case["causal"],
                            return_lse=case["lse"])
    tq, hq, d = q.shape
    tk, hk, _ = k.shape
    group = hq // hk
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    at_q, at_k = torch.arange(tq, device=q.device), torch.arange(tk, device=q.device)
    seq_q = torch.searchsorted(cu_q[1:], at_q, right=True)
    seq_k = torch.searchsorted(cu_k[1:], at_k, right=True)
    allowed = seq_q[:, None] == seq_k[None, :]
    if case["causal"]:
        # counted from the sequences' ends: the last query sees the last key
        allowed &= (at_k - cu_k[seq_k + 1])[None, :] <= (at_q - cu_q[seq_q + 1])[:, None]
    q32 = q.float().view(tq, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * tq, d)
    k32 = k.float().permute(1, 2, 0).contiguous()
    v32 = v.float().permute(1, 0, 2).contiguous()
    s = torch.bmm(q32, k32).mul_(d ** -0.5).view(hk, group, tq, tk)
    s.masked_fill_(~allowed, float("-inf"))
    top = s.amax(dim=-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.bmm(p.view(hk, group * tq, tk), v32).view(hk, group, tq, d)
    o = torch.where(total > 0, o / total, 0.0).permute(2, 0, 1, 3).reshape(tq, hq, d).to(q.dtype)
    if not case["lse"]:
        return o
    return o, (top + total.log()).view(hq, tq).t().contiguous()


def _activation(z, act):
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z)) if act == "silu" else z


def _run_linear(st):
    case, x, gate, residual = st["case"], st["x"], st["gate"], st["residual"]
    if own:
        import bit_quantized_diffusion_amd as bq
        return bq.linear16(x, st["w"], st["bias"], activation=case["act"], gate=gate, residual=residual,
                           group_rows=st["group_rows"])
    y = _activation(x.float() @ st["w"].float().t() + st["bias"].float(), case["act"])
    if gate is not None:
        y = (y.view(gate.shape[0], -1, y.shape[1]) * gate.float()[:, None, :]).view_as(y)
    if residual is not None:
        y = y + residual.float()
    return y.to(x.dtype)


def _run_norm(st):
    x, weight, bias, scale, shift = st["x"], st["weight"], st["bias"], st["scale"], st["shift"]
    if own:
        import bit_quantized_diffusion_amd as bq
        return bq.layer_norm(x, weight, bias, scale=scale, shift=shift, group_rows=st["group_rows"], eps=1e-6)
    x32 = x.float()
    off = x32 - x32.mean(dim=1, keepdim=True)
    y = off * torch.rsqrt((off * off).mean(dim=1, keepdim=True) + 1e-6)
    if weight is not None:
        y = y * weight.float() + bias.float()
    if scale is not None:
        y = y.view(scale.shape[0], -1, y.shape[1]) * (1.0 + scale.float())[:, None, :] + shift.float()[:, None, :]
    return y.view_as(x32).to(x.dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "attention":
        lens_q, lens_k = _lens(case["lens_q"]), _lens(case["lens_k"])
        hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
        pairs = 0
        for nq, nk in zip(lens_q, lens_k):
            if not case["causal"]:
                pairs += nq * nk
            else:  # query i sees max(0, i + 1 + nk - nq) keys
                first = max(1, nk - nq + 1)
                pairs += (first + nk) * (nk - first + 1) // 2 if nk >= first else 0
        moved = 2 * d * (2 * sum(lens_q) * hq + 2 * sum(lens_k) * hk) + (4 * sum(lens_q) * hq if case["lse"] else 0)
        return {"bytes": moved, "flops": 4 * d * hq * pairs}
    m, k = case["m"], case["k"]
    if case["op"] == "linear":
        n = case["n"]
        vectors = n * (1 + (case["groups"] if case["gate"] else 0))
        return {"bytes": 2 * (m * k + n * k + m * n * (2 if case["residual"] else 1) + vectors), "flops": 2 * m * n * k}
    vectors = k * ((2 if case["affine"] else 0) + (2 * case["groups"] if case["modulate"] else 0))
    return {"bytes": 2 * (2 * m * k + vectors), "flops": 8 * m * k}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attention":
        q, k, v = (st[name].double() for name in "qkv")
        group, d = case["heads_q"] // case["heads_k"], case["head_dim"]
        out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
        q0 = k0 = 0
        for nq, nk in zip(_lens(case["lens_q"]), _lens(case["lens_k"])):
            for h in range(case["heads_q"] if nq and nk else 0):
                keys, values = k[k0:k0 + nk, h // group], v[k0:k0 + nk, h // group]
                scores = (q[q0:q0 + nq, h] @ keys.T) / math.sqrt(d)
                if case["causal"]:
                    last = torch.arange(nq, device=q.device) + (nk - nq)
                    scores[torch.arange(nk, device=q.device)[None, :] > last[:, None]] = -math.inf
                row = torch.logsumexp(scores, dim=1)
                lse[q0:q0 + nq, h] = row
                weights = torch.exp(scores - torch.where(torch.isinf(row), torch.zeros_like(row), row)[:, None])
                out[q0:q0 + nq, h] = weights @ values
            q0, k0 = q0 + nq, k0 + nk
        return (out, lse) if case["lse"] else out
    x = st["x"].double()
    group_of = torch.arange(case["m"], device=x.device) // st["group_rows"]
    if case["op"] == "linear":
        z = torch.addmm(st["bias"].double(), x, st["w"].double().T)
        if case["act"] == "gelu":
            z = torch.nn.functional.gelu(z, approximate="tanh")
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        if st["gate"] is not None:
            z = z * st["gate"].double()[group_of]
        return z if st["residual"] is None else z + st["residual"].double()
    y = (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + 1e-6)
    if st["weight"] is not None:
        y = torch.addcmul(st["bias"].double(), y, st["weight"].double())
    if st["scale"] is not None:
        y = torch.addcmul(st["shift"].double()[group_of], y, 1.0 + st["scale"].double()[group_of])
    return y
