"""Measured cases of the operators around the block-FP8 linear layer.

Five operators, the parts of a served decoder between its linear layers:

* ``norm``    residual addition, RMS norm and 1x128 E4M3 quantisation
              (``fp8act.fp8_rmsnorm_quant``);
* ``silu``    silu(gate) * up and 1x128 E4M3 quantisation
              (``fp8act.fp8_silu_mul_quant``);
* ``append``  new keys and values quantised into a paged E4M3 cache
              (``fp8act.fp8_kv_append``);
* ``attend``  attention of the new tokens over that cache
              (``fp8act.fp8_kv_attention``);
* ``verify``  acceptance of drafted tokens against the target's logits and the
              draw of the next token (``fp8act.verify_drafts``).

Each has a plain form in elementary torch operations (fp32, rounded once) and
its definition in 64 bits (``exact``). E4M3 codes are returned as float8
tensors, that is as the values they stand for.
"""
from __future__ import annotations

import math

import torch

own = False

G = 128          # quantisation group of the linear layers
E4M3_MAX = 448.0
EPS = 1e-6
DEV = "cuda"

# Sizes: hidden 5120, MLP 2 x 8704 and the 151936-token vocabulary are this
# library's projection shapes; 24 query and 4 key/value heads of 128 are the
# (5120, 3072) output projection's input. 34 sequences x 3 tokens is its
# batched decode with two drafted tokens, 8 tokens its longest verify step,
# 4096 its prefill chunk.
HIDDEN, MLP, VOCAB = 5120, 8704, 151936


def listed():
    return [
        # one decoded token, where launch and reduction latency are all there is
        {"name": "norm decode", "op": "norm", "M": 1, "K": HIDDEN, "residual": True},
        # a prefill chunk: bandwidth
        {"name": "norm prefill", "op": "norm", "M": 4096, "K": HIDDEN, "residual": True},
        # the 8 tokens of the longest verify step
        {"name": "silu verify", "op": "silu", "M": 8, "I": MLP},
        # a prefill chunk: bandwidth and the exponential's rate
        {"name": "silu prefill", "op": "silu", "M": 4096, "I": MLP},
        # 34 sequences x 3 tokens scattered over pages
        {"name": "append batch", "op": "append", "T": 102, "H": 4, "D": 128, "page": 64},
        # a prefill chunk written page after page
        {"name": "append prefill", "op": "append", "T": 4096, "H": 4, "D": 128, "page": 64},
        # one request, one token, a short context: latency
        {"name": "attend decode", "op": "attend", "B": 1, "n": 1, "L": 4096, "ragged": False, "H": 4, "group": 6,
         "D": 128, "page": 64},
        # one request, the 8 tokens of a verify step, a long context: bandwidth with 48 rows a head
        {"name": "attend verify long", "op": "attend", "B": 1, "n": 8, "L": 131072, "ragged": False, "H": 4,
         "group": 6, "D": 128, "page": 64},
        # 34 sequences of unequal lengths x 3 tokens: balance
        {"name": "attend batch ragged", "op": "attend", "B": 34, "n": 3, "L": 16384, "ragged": True, "H": 4,
         "group": 6, "D": 128, "page": 16},
        # a chunk of a prompt over what is cached of it: arithmetic
        {"name": "attend chunk", "op": "attend", "B": 1, "n": 512, "L": 16384, "ragged": False, "H": 4, "group": 6,
         "D": 128, "page": 64},
        # one request with 7 drafted tokens
        {"name": "verify single", "op": "verify", "B": 1, "k": 7, "V": VOCAB, "f32": False, "greedy_draft": False},
        # 34 sequences with 2 drafted tokens each
        {"name": "verify batch", "op": "verify", "B": 34, "k": 2, "V": VOCAB, "f32": False, "greedy_draft": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "silu", "append", "attend", "attend", "verify"])
    if op == "norm":
        return {"op": op, "M": _log_int(rng, 1, 4096), "K": G * _log_int(rng, 1, 40), "residual": rng.random() < 0.75}
    if op == "silu":
        return {"op": op, "M": _log_int(rng, 1, 4096), "I": G * _log_int(rng, 1, 68)}
    if op == "append":
        H, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256])
        return {"op": op, "T": _log_int(rng, 1, 4096 * 512 // max(512, H * D)), "H": H, "D": D,
                "page": rng.choice([16, 32, 64, 128])}
    if op == "attend":
        H, D, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 6, 8, 12])
        n = rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(2, 8), _log_int(rng, 9, 256)])
        B = _log_int(rng, 1, 48) if n <= 8 else 1
        # cached bytes below the long verify case's, scores below the chunk's
        most = min(131072 * 4 * 128 // (B * H * D), 512 * 24 * 16384 // (B * n * H * group))
        return {"op": op, "B": B, "n": n, "L": _log_int(rng, min(max(n, 16), most), most), "ragged": rng.random() < 0.6,
                "H": H, "group": group, "D": D, "page": rng.choice([16, 32, 64, 128])}
    k, f32 = rng.randint(1, 7), rng.random() < 0.3
    rows = 34 * 7 // (2 * k + 3) // (2 if f32 else 1)  # logits read below the batch case's
    return {"op": op, "B": _log_int(rng, 1, rows), "k": k, "V": _log_int(rng, 1000, VOCAB), "f32": f32,
            "greedy_draft": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(shape, g, dtype=torch.bfloat16):
    """N(0, 1) with one entry in a thousand twenty times larger, as hidden states have them."""
    x = torch.randn(shape, device=DEV, generator=g)
    x *= torch.where(torch.rand(shape, device=DEV, generator=g) < 0.001, 20.0, 1.0)
    return x.to(dtype)


def _lens(c, g):
    """Cached tokens per sequence, the new ones included."""
    if not c["ragged"]:
        return torch.full((c["B"],), c["L"], device=DEV, dtype=torch.int32)
    low = min(c["n"], c["L"])
    u = torch.rand(c["B"], device=DEV, generator=g)
    lens = (low * (c["L"] / low) ** u).round().to(torch.int32).clamp_(low, c["L"])
    lens[0] = c["L"]
    return lens


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"op": op, "case": case}
    if op == "norm":
        M, K = case["M"], case["K"]
        s["x"] = _activations((M, K), g)
        s["residual"] = (4.0 * torch.randn((M, K), device=DEV, generator=g)).bfloat16() if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(K, device=DEV, generator=g)).bfloat16()
        s["q"] = torch.empty((M, K), device=DEV, dtype=torch.float8_e4m3fn)
        s["sa"] = torch.empty((M, K // G), device=DEV)
        s["out"] = torch.empty((M, K), device=DEV, dtype=torch.bfloat16) if case["residual"] else None
    elif op == "silu":
        M, n = case["M"], case["I"]
        s["gate_up"] = (2.0 * torch.randn((M, 2 * n), device=DEV, generator=g)).bfloat16()
        s["q"] = torch.empty((M, n), device=DEV, dtype=torch.float8_e4m3fn)
        s["sa"] = torch.empty((M, n // G), device=DEV)
    elif op == "append":
        T, H, D, page = case["T"], case["H"], case["D"], case["page"]
        pages = -(-T // page) + 7
        # keys and values are columns of the fused projection's rows
        qkv = _activations((T, 3 * H * D), g)
        s["k"] = qkv[:, H * D:2 * H * D].unflatten(1, (H, D))
        s["v"] = qkv[:, 2 * H * D:].unflatten(1, (H, D))
        order = torch.randperm(pages, device=DEV, generator=g)
        at = torch.arange(T, device=DEV)
        if T <= 512:  # decode: every token goes to a place of its own
            at = torch.randperm(pages * page, device=DEV, generator=g)[:T]
            s["slots"] = at
        else:         # a prompt: in order, page after page
            s["slots"] = order[at // page] * page + at % page
        s["cache"] = (torch.zeros((pages, H, page, D), device=DEV, dtype=torch.uint8),
                      torch.zeros((pages, H, page, D), device=DEV, dtype=torch.uint8),
                      torch.ones((pages, H, page), device=DEV), torch.ones((pages, H, page), device=DEV))
    elif op == "attend":
        B, n, L, H, D, page = (case[k] for k in ("B", "n", "L", "H", "D", "page"))
        lens = _lens(case, g)
        per = -(-L // page)
        pages = B * per + 3
        s["table"] = torch.randperm(pages, device=DEV, generator=g)[:B * per].view(B, per).to(torch.int32)
        s["lens"] = lens
        s["cu_q"] = torch.arange(B + 1, device=DEV, dtype=torch.int32) * n
        s["q"] = torch.randn((B * n, H * case["group"], D), device=DEV, generator=g).bfloat16()
        cache = []
        for scale in (1.5, 1.0):  # keys, values: E4M3 of normals, an amax / 448 scale per token and head
            x = scale * torch.randn((pages, H, page, D), device=DEV, generator=g)
            f = x.abs().amax(-1, keepdim=True) / E4M3_MAX
            cache += [(x / f).to(torch.float8_e4m3fn).view(torch.uint8), f.squeeze(-1)]
            del x
        # slots that no token has written yet hold what was there before: NaN, say
        at = torch.arange(per * page, device=DEV).view(1, per, page)
        b, p, o = torch.nonzero(at >= lens.view(B, 1, 1), as_tuple=True)
        for t, bad in zip(cache, (0x7F, math.nan, 0xFF, math.nan)):
            t[s["table"][b, p].long(), :, o] = bad
        s["cache"] = (cache[0], cache[2], cache[1], cache[3])
        s["max_n"] = n
        s["out"] = torch.empty_like(s["q"])
    else:
        B, k, V = case["B"], case["k"], case["V"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        # a peaked target and a draft model that follows it with errors of its own
        t = 2.5 * torch.randn((B, k + 1, V), device=DEV, generator=g)
        t += torch.where(torch.rand((B, k + 1, V), device=DEV, generator=g) < 4.0 / V, 12.0, 0.0)
        d = t[:, :k] + 0.5 * torch.randn((B, k, V), device=DEV, generator=g)
        # one target in eight was cut to its likely tokens before: the others are -inf
        cut = torch.rand((B, k + 1, 1), device=DEV, generator=g) < 0.125
        t = torch.where(cut & (t < 2.0), -math.inf, t)
        s["target"], s["draft"] = t.to(dt), d.to(dt)
        temp = 0.6 + 0.6 * torch.rand(B, device=DEV, generator=g)
        race = torch.empty((B, k, V), device=DEV).exponential_(generator=g)
        drawn = (s["draft"].float() / temp.view(B, 1, 1)).softmax(-1) / race
        if case["greedy_draft"]:
            drawn, s["draft"] = s["draft"].float(), None
        s["tokens"] = drawn.argmax(-1).to(torch.int32)
        s["uniform"] = torch.rand((B, k), device=DEV, generator=g)
        s["noise"] = torch.empty((B, V), device=DEV).exponential_(generator=g).clamp_(min=1e-20)
        temp[1::5] = 0.0  # some sequences are decoded greedily
        s["temperature"] = temp
    return s


# ------------------------------------------------------------- plain forms
def _quant(y):
    """fp32 [M, K] -> E4M3 codes and one amax / 448 scale per 128 columns."""
    M, K = y.shape
    y = y.view(M, K // G, G)
    amax = y.abs().amax(-1)
    sa = torch.where(amax == 0, 1.0, amax / E4M3_MAX)
    q = (y / sa.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(M, K), sa


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    q, sa = _quant(y)
    out = {"q": q, "sa": sa}
    if s["residual"] is not None:
        out["residual"] = h.bfloat16()
    return out


def _plain_silu(s):
    gate, up = s["gate_up"].float().chunk(2, -1)
    q, sa = _quant(gate / (1.0 + torch.exp(-gate)) * up)
    return {"q": q, "sa": sa}


def _plain_append(s):
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    for x, codes, scales in ((s["k"], s["cache"][0], s["cache"][2]), (s["v"], s["cache"][1], s["cache"][3])):
        x = x.float()
        amax = x.abs().amax(-1)
        f = torch.where(amax == 0, 1.0, amax / E4M3_MAX)
        q = (x / f.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        codes[at, :, off] = q.view(torch.uint8)
        scales[at, :, off] = f
    return _cache_out(s)


def _cache_out(s):
    k, v, ks, vs = s["cache"]
    return {"k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn), "k_scale": ks, "v_scale": vs}


def _plain_attend(s):
    c = s["case"]
    B, n, H, D = c["B"], c["n"], c["H"], c["D"]
    k8, v8, ks, vs = s["cache"]
    at = s["table"].long()
    L = at.shape[1] * c["page"]
    pos = torch.arange(L, device=DEV)
    there = (pos < s["lens"].view(B, 1)).view(B, 1, L, 1)

    def read(codes, scales):  # [B, H, L, D] in fp32, zero where nothing was written
        x = codes.view(torch.float8_e4m3fn)[at].float() * scales[at].unsqueeze(-1)
        return torch.where(there, x.transpose(1, 2).reshape(B, H, L, D), 0.0)

    q = s["q"].float().view(B, n, H, c["group"], D).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(q.reshape(B, H, -1, D), read(k8, ks).transpose(2, 3)).view(B, H, c["group"], n, L)
    scores *= D ** -0.5
    last = s["lens"].view(B, 1) - n + torch.arange(n, device=DEV)  # the last position that new token i sees
    seen = (pos <= last.unsqueeze(-1)).view(B, 1, 1, n, L)
    scores = torch.where(seen, scores, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, -1, L), read(v8, vs)).view(B, H, c["group"], n, D)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B * n, H * c["group"], D).bfloat16()


def _softmax(logits, temperature):
    """Softmax of logits / temperature along the last axis; all zero where every logit is -inf."""
    x = logits / torch.where(temperature > 0, temperature, 1.0).view(-1, 1, 1)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0)


def _verify(s, dtype):
    """The definition of the verification in `dtype`."""
    B, k, V = s["case"]["B"], s["case"]["k"], s["case"]["V"]
    temp, tokens = s["temperature"].to(dtype), s["tokens"].long()
    target, ids = s["target"].to(dtype), torch.arange(V, device=DEV)
    p = _softmax(target, temp)
    top = torch.where((target == target.amax(-1, keepdim=True)) & (target > -math.inf), ids, V).amin(-1, keepdim=True)
    p = torch.where((temp > 0).view(B, 1, 1), p, (ids == top).to(dtype))
    point = (ids == tokens.unsqueeze(-1)).to(dtype)
    q = point if s["draft"] is None else _softmax(s["draft"].to(dtype), temp)
    q = torch.where((temp > 0).view(B, 1, 1), q, point)
    px, qx = p[:, :k].gather(2, tokens.unsqueeze(-1)).squeeze(-1), q.gather(2, tokens.unsqueeze(-1)).squeeze(-1)
    prob = torch.where(qx > 0, (px / qx).clamp(max=1.0), (px > 0).to(dtype))
    took = (s["uniform"].to(dtype) < prob).to(torch.int64).cumprod(-1).sum(-1)
    row = torch.arange(B, device=DEV)
    p_at, q_at = p[row, took], q[row, took.clamp(max=k - 1)]
    rest = torch.where((took < k).view(B, 1), (p_at - q_at).clamp(min=0), p_at)
    rest = torch.where((rest > 0).any(-1, keepdim=True) & (temp > 0).view(B, 1), rest, p_at)
    key = rest / s["noise"].to(dtype)
    best = torch.where((key == key.amax(-1, keepdim=True)) & (rest > 0), ids, V).amin(-1)
    best = torch.where(best < V, best, -1)
    j = torch.arange(k + 1, device=DEV)
    padded = torch.cat([tokens, tokens[:, :1]], 1)
    out = torch.where(j < took.view(B, 1), padded, torch.where(j == took.view(B, 1), best.view(B, 1), -1))
    return took.to(torch.int32), out.to(torch.int32), prob


def run(s):
    op = s["op"]
    if own:
        from block_scaled_fp8_act_gb300 import fp8act
        if op == "norm":
            got = fp8act.fp8_rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS, q=s["q"], sa=s["sa"],
                                           residual_out=s["out"])
            return dict(zip(("q", "sa", "residual"), got))
        if op == "silu":
            q, sa = fp8act.fp8_silu_mul_quant(s["gate_up"], q=s["q"], sa=s["sa"])
            return {"q": q, "sa": sa}
        if op == "append":
            fp8act.fp8_kv_append(s["k"], s["v"], s["slots"], s["cache"])
            return _cache_out(s)
        if op == "attend":
            return fp8act.fp8_kv_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu_q"], max_q_len=s["max_n"],
                                           out=s["out"])
        took, tokens, prob = fp8act.verify_drafts(s["target"], s["tokens"], s["uniform"], s["noise"], s["temperature"],
                                                  draft_logits=s["draft"])
        return {"accepted": took, "tokens": tokens, "prob": prob}
    if op == "verify":
        took, tokens, prob = _verify(s, torch.float32)
        return {"accepted": took, "tokens": tokens, "prob": prob}
    return {"norm": _plain_norm, "silu": _plain_silu, "append": _plain_append, "attend": _plain_attend}[op](s)


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "norm":
        e = case["M"] * case["K"]
        return {"bytes": e * (7 if case["residual"] else 3) + 4 * e // G + 2 * case["K"], "flops": 8 * e}
    if op == "silu":
        e = case["M"] * case["I"]
        return {"bytes": 5 * e + 4 * e // G, "flops": 8 * e}
    if op == "append":
        h = case["T"] * case["H"]
        return {"bytes": h * (6 * case["D"] + 8) + 8 * case["T"], "flops": 6 * h * case["D"]}
    if op == "attend":
        B, n, H, D, hq = case["B"], case["n"], case["H"], case["D"], case["H"] * case["group"]
        low = min(n, case["L"])
        # the mean of lengths spread evenly over their logarithm, the first one the longest
        mean = (case["L"] - low) / math.log(case["L"] / low) if case["ragged"] and case["L"] > low else case["L"]
        total = case["L"] + (B - 1) * mean
        return {"bytes": int(total * H * (2 * D + 8)) + 4 * B * n * hq * D,
                "flops": int(4 * n * hq * D * max(total - B * (n - 1) / 2, total / 2))}
    B, k, V = case["B"], case["k"], case["V"]
    rows = k + 1 + (0 if case["greedy_draft"] else k)
    return {"bytes": B * V * (rows * (4 if case["f32"] else 2) + 4), "flops": 4 * B * rows * V}


# ----------------------------------------------------- definition, 64 bits
def _e4m3(x):
    """The nearest E4M3 value of a 64-bit one, ties to the even significand, saturating."""
    a = x.abs().clamp(max=E4M3_MAX)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3.0)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _scaled(y):
    amax = y.abs().amax(-1, keepdim=True)
    f = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    return _e4m3(y / f), f.squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("norm", "silu"):
        if op == "norm":
            h = s["x"].double()
            h = h if s["residual"] is None else h + s["residual"].double()
            y = s["weight"].double() * h / torch.sqrt(torch.square(h).sum(-1, keepdim=True) / h.shape[-1] + EPS)
        else:
            n = case["I"]
            gate, up = s["gate_up"][:, :n].double(), s["gate_up"][:, n:].double()
            y = up * gate * torch.sigmoid(gate)
        q, f = _scaled(y.unflatten(-1, (-1, G)))
        out = {"q": q.flatten(-2), "sa": f}
        if op == "norm" and s["residual"] is not None:
            out["residual"] = h
        return out
    if op == "append":
        page = case["page"]
        out = {}
        for name, x, codes, scales in (("k", s["k"], s["cache"][0], s["cache"][2]),
                                       ("v", s["v"], s["cache"][1], s["cache"][3])):
            q, f = _scaled(x.double())
            values, new = codes.view(torch.float8_e4m3fn).double(), scales.double()
            values[s["slots"] // page, :, s["slots"] % page] = q
            new[s["slots"] // page, :, s["slots"] % page] = f
            out[name], out[name + "_scale"] = values, new
        return out
    if op == "attend":
        B, n, H, D, page, group = (case[k] for k in ("B", "n", "H", "D", "page", "group"))
        out = torch.zeros((B, n, H, group, D), device=DEV, dtype=torch.float64)
        q = s["q"].double().view(B, n, H, group, D)
        for b in range(B):
            L = int(s["lens"][b])
            at = s["table"][b, :-(-L // page)].long()
            for h in range(H):
                k, v = ((s["cache"][i][at, h].view(torch.float8_e4m3fn).double()
                         * s["cache"][i + 2][at, h].double().unsqueeze(-1)).flatten(0, 1)[:L] for i in (0, 1))
                x = torch.einsum("ngd,ld->ngl", q[b, :, h], k) / math.sqrt(D)
                hidden = torch.arange(L, device=DEV) > (L - n + torch.arange(n, device=DEV)).view(n, 1, 1)
                x = x.masked_fill(hidden, -math.inf)
                out[b, :, h] = torch.einsum("ngl,ld->ngd", torch.softmax(x, -1).nan_to_num(0.0), v)
        return out.view(B * n, H * group, D)
    return {"accepted": None, "tokens": None, "prob": _verify_prob(s)}


def _verify_prob(s):
    """Acceptance probabilities min(1, p(x) / q(x)) from logarithms, in 64 bits."""
    B, k = s["tokens"].shape
    tokens, temp = s["tokens"].long().unsqueeze(-1), s["temperature"].double().view(B, 1, 1)
    target = s["target"][:, :k].double()
    lp = torch.log_softmax(target / temp.clamp(min=0.1), -1).gather(2, tokens)
    lq = torch.zeros_like(lp)
    if s["draft"] is not None:
        lq = torch.log_softmax(s["draft"].double() / temp.clamp(min=0.1), -1).gather(2, tokens)
    first = (target == target.amax(-1, keepdim=True)).to(torch.int8).argmax(-1, keepdim=True) == tokens
    return torch.where(temp > 0, torch.exp((lp - lq).clamp(max=0.0)), first.double()).squeeze(-1)
