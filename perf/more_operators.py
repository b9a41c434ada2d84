"""Measured cases of the operators around the paged E4M3 cache.

Four operators, what a decoder layer does with its cache beside appending to it
and plain causal attention:

* ``rope``   RMS norms of the query and key heads, rotary positions of one or
             several axes, keys and values quantised into the cache
             (``fp8act.fp8_rope_append``);
* ``attend`` attention over the cache with capped scores, a distance bias, a
             window, a prefix or documents (``fp8act.fp8_kv_attention`` with
             a score function);
* ``mass``   the attention weight that every cached token gets, added up
             (``fp8act.fp8_kv_attention_mass``);
* ``evict``  the tokens of most weight into fresh pages
             (``fp8act.fp8_kv_evict``).

Each has a plain form in elementary torch operations (fp32, angles in 64 bits,
rounded once) and its definition in 64 bits (``exact``). E4M3 codes are returned
as float8 tensors, that is as the values they stand for.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
DEV = "cuda"


# Sizes: 24 query and 4 key/value heads of 128 are this library's output
# projection's; 34 sequences x 3 tokens is its batched decode with two drafted
# tokens, 8 tokens its longest verify step, 4096 its prefill chunk.
def _rope(name, **kw):
    return {"name": name, "op": "rope", "T": 1, "heads": 24, "H": 4, "D": 128, "rot": 128, "axes": 1, "norm": True,
            "interleaved": False, "page": 64, **kw}


def _attend(name, **kw):
    return {"name": name, "op": "attend", "B": 1, "n": 1, "L": 4096, "ragged": False, "H": 4, "group": 6, "D": 128,
            "page": 64, "cap": 0.0, "window": 0, "prefix": 0, "doc": 0, "bias": False, **kw}


def _mass(name, **kw):
    return {"name": name, "op": "mass", "B": 1, "n": 1, "L": 4096, "ragged": False, "H": 4, "group": 6, "D": 128,
            "page": 64, "cap": 0.0, "window": 0, "prefix": 0, "doc": 0, "bias": False, "add": True, **kw}


def _evict(name, **kw):
    return {"name": name, "op": "evict", "B": 1, "L": 2048, "ragged": False, "keep": 1024, "recent": 64, "first": 4,
            "H": 4, "D": 128, "page": 64, **kw}


def listed():
    return [
        # one decoded token: launch and latency are all there is
        _rope("rope decode"),
        # 34 sequences x 3 tokens, half of a head rotated
        _rope("rope batch", T=102, rot=64),
        # a prefill chunk with images in it (time, height and width positions): bandwidth
        _rope("rope prefill", T=4096, axes=3),
        # one token of a layer with a sliding window and capped scores: latency
        _attend("attend window", L=16384, cap=50.0, window=1024),
        # 34 sequences of unequal lengths x 3 tokens, a long window and capped scores: balance
        _attend("attend batch capped", B=34, n=3, L=16384, ragged=True, page=16, cap=30.0, window=4096),
        # the 8 tokens of a verify step over a long context, weights that fall with the distance
        _attend("attend verify bias", n=8, L=131072, bias=True),
        # a chunk of a prompt of several documents behind a prefix that all may see: arithmetic
        _attend("attend chunk prefix", n=512, L=16384, prefix=2048, doc=4096, cap=50.0),
        # one decoded token of each of 34 sequences, added to what there is: bandwidth
        _mass("mass batch", B=34, L=16384, ragged=True, page=16),
        # the last 32 tokens of a long prompt say which of its tokens matter: arithmetic
        _mass("mass prompt", n=32, L=131072, add=False),
        # a short cache cut in half: latency
        _evict("evict short"),
        # a long prompt cut to a sixteenth
        _evict("evict prompt", L=131072, keep=8192, recent=256),
        # 34 sequences of unequal lengths cut to 4096 tokens: bandwidth
        _evict("evict batch", B=34, L=16384, ragged=True, keep=4096, page=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "mass", "evict"])
    H, D, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    if op == "rope":
        group = rng.choice([1, 2, 3, 4, 6, 8, 12])
        most = max(1, 4096 * 32 * 128 // max(32 * 128, (group + 2) * H * D))
        return {"op": op, "T": _log_int(rng, 1, most), "heads": group * H, "H": H, "D": D,
                "rot": rng.choice([D, D, D // 2, D // 4, 16 * rng.randint(1, D // 16)]), "axes": rng.randint(1, 4),
                "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.3, "page": page}
    if op == "evict":
        B = _log_int(rng, 1, 48)
        most = 131072 * 4 * 128 // (B * H * D)
        L = _log_int(rng, 16, most)
        keep = _log_int(rng, 1, max(1, min(L, most // 2)))
        return {"op": op, "B": B, "L": L, "ragged": rng.random() < 0.6, "keep": keep,
                "recent": rng.randint(0, keep // 2), "first": rng.randint(0, min(4, keep // 2)), "H": H, "D": D, "page": page}
    group = rng.choice([1, 2, 3, 4, 6, 8, 12])
    n = rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(2, 8), _log_int(rng, 9, 256)])
    B = _log_int(rng, 1, 48) if n <= 8 else 1
    # cached bytes and scores below the largest listed cases'
    most = min(131072 * 4 * 128 // (B * H * D), 512 * 24 * 16384 // (B * n * H * group))
    if op == "mass":
        most = min(most, 32 * 24 * 131072 // (B * n * H * group))
    L = _log_int(rng, min(max(n, 16), most), most)
    case = {"op": op, "B": B, "n": n, "L": L, "ragged": rng.random() < 0.6, "H": H, "group": group, "D": D, "page": page,
            "cap": rng.choice([0.0, 0.0, 20.0, 50.0]), "window": rng.choice([0, _log_int(rng, 1, L)]),
            "prefix": rng.choice([0, 0, _log_int(rng, 1, L)]), "doc": rng.choice([0, 0, _log_int(rng, 1, L)]),
            "bias": rng.random() < 0.4}
    if op == "mass":
        case["add"] = rng.random() < 0.7
    elif not (case["cap"] or case["window"] or case["prefix"] or case["doc"] or case["bias"]):
        case["cap"] = 30.0
    return case


# ------------------------------------------------------------------ inputs
def _lens(c, g, low):
    """Cached tokens per sequence, the new ones included."""
    if not c["ragged"]:
        return torch.full((c["B"],), c["L"], device=DEV, dtype=torch.int32)
    low = min(low, c["L"])
    u = torch.rand(c["B"], device=DEV, generator=g)
    lens = (low * (c["L"] / low) ** u).round().to(torch.int32).clamp_(low, c["L"])
    lens[0] = c["L"]
    return lens


def _paged(c, g, lens, extra):
    """A page table and a cache of `extra` more pages: E4M3 of normals with an amax / 448 scale per token and head."""
    B, H, D, page = (c[k] for k in ("B", "H", "D", "page"))
    per = -(-c["L"] // page)
    pages = B * per + extra
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    table = order[:B * per].view(B, per)
    cache = []
    for scale in (1.5, 1.0):  # keys, values
        x = scale * torch.randn((pages, H, page, D), device=DEV, generator=g)
        f = x.abs().amax(-1, keepdim=True) / E4M3_MAX
        cache += [(x / f).to(torch.float8_e4m3fn).view(torch.uint8), f.squeeze(-1)]
        del x
    # slots that no token has written yet hold what was there before: NaN, say
    at = torch.arange(per * page, device=DEV).view(1, per, page)
    b, p, o = torch.nonzero(at >= lens.view(B, 1, 1), as_tuple=True)
    for t, bad in zip(cache, (0x7F, math.nan, 0xFF, math.nan)):
        t[table[b, p].long(), :, o] = bad
    return table, order[B * per:], (cache[0], cache[2], cache[1], cache[3])


def _prepare_rope(case, g):
    T, heads, H, D, rot, page = (case[k] for k in ("T", "heads", "H", "D", "rot", "page"))
    s = {}
    # queries, keys and values are columns of the fused projection's rows
    qkv = torch.randn((T, (heads + 2 * H) * D), device=DEV, generator=g)
    qkv = (qkv * torch.where(torch.rand(qkv.shape, device=DEV, generator=g) < 0.001, 20.0, 1.0)).bfloat16()
    s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split([heads * D, H * D, H * D], 1))
    s["q_weight"], s["k_weight"] = ((1.0 + 0.2 * torch.randn(D, device=DEV, generator=g)).bfloat16() if case["norm"] else None
                                    for _ in range(2))
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    s["inv_freq"] = 1e6 ** (-2.0 * i / rot)
    axes = case["axes"]
    # somewhere in a long context; with several axes, places in an image that starts there
    start = int(torch.randint(0, 262144, (1,), device=DEV, generator=g))
    pos = (start + torch.arange(T, device=DEV)).repeat(axes, 1)
    if axes > 1:
        pos[1:] = start + torch.randint(0, 128, (axes - 1, T), device=DEV, generator=g)
    s["positions"] = pos
    s["axes"] = (i.long() % axes).to(torch.int32) if axes > 1 else None  # the axes take the frequencies in turn
    pages = -(-T // page) + 7
    order = torch.randperm(pages, device=DEV, generator=g)
    at = torch.arange(T, device=DEV)
    if T <= 512:  # decode: every token goes to a place of its own
        s["slots"] = torch.randperm(pages * page, device=DEV, generator=g)[:T]
    else:         # a prompt: in order, page after page
        s["slots"] = order[at // page] * page + at % page
    s["cache"] = (torch.zeros((pages, H, page, D), device=DEV, dtype=torch.uint8),
                  torch.zeros((pages, H, page, D), device=DEV, dtype=torch.uint8),
                  torch.ones((pages, H, page), device=DEV), torch.ones((pages, H, page), device=DEV))
    s["out"] = torch.empty((T, heads, D), device=DEV, dtype=torch.bfloat16)
    return s


def _prepare_rows(case, g):
    """What attention and its mass have in common."""
    B, n, L, H, D = (case[k] for k in ("B", "n", "L", "H", "D"))
    lens = _lens(case, g, case["n"])
    s = {"lens": lens, "max_n": n, "cu_q": torch.arange(B + 1, device=DEV, dtype=torch.int32) * n}
    s["table"], _, s["cache"] = _paged(case, g, lens, 3)
    s["q"] = torch.randn((B * n, H * case["group"], D), device=DEV, generator=g).bfloat16()
    s["prefix"] = s["first"] = s["slopes"] = None
    if case["prefix"]:
        s["prefix"] = torch.randint(0, case["prefix"] + 1, (B,), device=DEV, generator=g).to(torch.int32)
        s["prefix"][0] = case["prefix"]
    if case["doc"]:
        starts = torch.rand((B, L), device=DEV, generator=g) < 1.0 / case["doc"]
        begin = torch.where(starts, torch.arange(L, device=DEV), 0).cummax(1).values
        at = (lens.view(B, 1).long() - n + torch.arange(n, device=DEV)).clamp(min=0)
        s["first"] = begin.gather(1, at).flatten().to(torch.int32)
    if case["bias"]:  # a geometric sequence over the heads
        heads = H * case["group"]
        s["slopes"] = 2.0 ** (-8.0 * (torch.arange(heads, device=DEV) + 1.0) / heads)
    return s


def prepare(case, seed):
    g, op = torch.Generator(device=DEV).manual_seed(seed), case["op"]
    if op == "rope":
        s = _prepare_rope(case, g)
    elif op == "attend":
        s = _prepare_rows(case, g)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device=DEV)
    elif op == "mass":
        s = _prepare_rows(case, g)
        x = _scores({**s, "case": case})
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        lse = (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))).squeeze(-1)  # what the attention before it left
        s["lse"] = lse.permute(0, 3, 1, 2).reshape(s["q"].shape[:2]).contiguous()
        s["mass"] = torch.rand(s["cache"][2].shape, device=DEV, generator=g) if case["add"] else torch.zeros_like(s["cache"][2])
    else:
        B, H, page = case["B"], case["H"], case["page"]
        lens = _lens(case, g, 16)
        per = -(-case["keep"] // page)
        s = {"lens": lens}
        s["table"], spare, s["cache"] = _paged(case, g, lens, B * per + 3)
        s["new_table"] = spare[:B * per].view(B, per).contiguous()
        # a few tokens have most of the weight, and some none that 32 bits can show
        mass = torch.exp(2.0 * torch.randn((s["cache"][2].shape), device=DEV, generator=g))
        s["mass"] = torch.where(torch.rand(mass.shape, device=DEV, generator=g) < 0.1, 0.0, mass)
        s["keep"] = torch.full((B,), case["keep"], device=DEV, dtype=torch.int32)
        s["new_lens"] = torch.empty(B, device=DEV, dtype=torch.int32)
        s["kept"] = torch.empty((B, H, per * page), device=DEV, dtype=torch.int32)
    s["op"], s["case"] = op, case
    return s


# ------------------------------------------------------------- plain forms
def _cache_out(s):
    k, v, ks, vs = s["cache"]
    return {"k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn), "k_scale": ks, "v_scale": vs}


def _head_norm(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_rope(s):
    page = s["case"]["page"]
    axis = torch.zeros(len(s["inv_freq"]), device=DEV, dtype=torch.long) if s["axes"] is None else s["axes"].long()
    angle = s["positions"][axis].T.double() * s["inv_freq"]  # [T, rot / 2]
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    q, k = (_rotate(_head_norm(s[x], s[x + "_weight"]), cos, sin, s["case"]["interleaved"]) for x in ("q", "k"))
    at, off = s["slots"] // page, s["slots"] % page

    def store(x, codes, scales):
        amax = x.abs().amax(-1)
        f = torch.where(amax == 0, 1.0, amax / E4M3_MAX)
        codes[at, :, off] = (x / f.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[at, :, off] = f

    store(k, s["cache"][0], s["cache"][2])
    store(s["v"].float(), s["cache"][1], s["cache"][3])
    return {"q": q.bfloat16(), **_cache_out(s)}


def _places(s):
    """Cached places [B, H, L] of the sequences' pages, and which of them hold a token [B, 1, L]."""
    L = s["table"].shape[1] * s["case"]["page"]
    pos = torch.arange(L, device=DEV)
    return pos, (pos < s["lens"].view(-1, 1)).unsqueeze(1)


def _read(s, codes, scales):
    """[B, H, L, D] in fp32, zero where nothing was written."""
    at, (_, there) = s["table"].long(), _places(s)
    x = codes.view(torch.float8_e4m3fn)[at].float() * scales[at].unsqueeze(-1)
    x = x.transpose(1, 2).flatten(2, 3)
    return torch.where(there.unsqueeze(-1), x, 0.0)


def _seen(s):
    """Which positions new token i of a sequence sees, [B, n, L], and their distance from it."""
    c, (pos, there) = s["case"], _places(s)
    B, n = c["B"], c["n"]
    own_pos = (s["lens"].view(B, 1) - n + torch.arange(n, device=DEV)).unsqueeze(-1)  # of the new tokens
    seen = pos <= own_pos
    if c["window"]:
        seen &= own_pos - pos < c["window"]
    if s["first"] is not None:
        seen &= pos >= s["first"].view(B, n, 1)
    if s["prefix"] is not None:
        seen |= (pos < s["prefix"].view(B, 1, 1)) & there
    return seen, (own_pos - pos).abs()


def _scores(s):
    """[B, H, group, n, L] in fp32, -inf where a token does not see a position."""
    c = s["case"]
    B, n, H, D = c["B"], c["n"], c["H"], c["D"]
    q = s["q"].float().view(B, n, H, c["group"], D).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(B, H, -1, D), _read(s, s["cache"][0], s["cache"][2]).transpose(2, 3))
    x = x.view(B, H, c["group"], n, -1) * D ** -0.5
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    seen, far = _seen(s)
    if s["slopes"] is not None:
        x = x - s["slopes"].view(H, c["group"], 1, 1) * far.view(B, 1, 1, n, -1).float()
    return torch.where(seen.view(B, 1, 1, n, -1), x, -math.inf)


def _plain_attend(s):
    c = s["case"]
    B, n, H, D = c["B"], c["n"], c["H"], c["D"]
    x = _scores(s)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, c["group"] * n, -1), _read(s, s["cache"][1], s["cache"][3])).view(B, H, c["group"], n, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total)).squeeze(-1)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B * n, -1, D).bfloat16(), "lse": lse.permute(0, 3, 1, 2).reshape(B * n, -1)}


def _plain_mass(s):
    c = s["case"]
    B, n, H, page = c["B"], c["n"], c["H"], c["page"]
    lse = s["lse"].view(B, n, H, c["group"]).permute(0, 2, 3, 1).unsqueeze(-1)
    p = torch.exp(_scores(s) - torch.where(lse == -math.inf, math.inf, lse))
    got = p.sum((2, 3))  # [B, H, L]
    pos, there = _places(s)
    # the new tokens' own places start from zero
    b, j = torch.nonzero(there.squeeze(1), as_tuple=True)
    at, off = s["table"][b, j // page].long(), j % page
    new = got[b, :, j]
    if c["add"]:
        new = new + torch.where((j < s["lens"][b] - n).unsqueeze(-1), s["mass"][at, :, off], 0.0)
    s["mass"][at, :, off] = new
    return s["mass"]


def _plain_evict(s):
    c = s["case"]
    B, H, page = c["B"], c["H"], c["page"]
    pos, there = _places(s)
    lens, keep = s["lens"].view(B, 1, 1).long(), s["keep"].view(B, 1, 1).long()
    mass = s["mass"][s["table"].long()].transpose(1, 2).flatten(2, 3)  # [B, H, L]
    recent = keep.clamp(max=c["recent"])
    first = torch.minimum(keep - recent, torch.full_like(keep, c["first"]))
    key = torch.where((pos >= lens - recent) | (pos < first), math.inf, mass)
    key = torch.where(there, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    count = torch.minimum(lens, keep)
    most = s["kept"].shape[2]
    slot = torch.arange(most, device=DEV)
    if order.shape[2] < most:
        order = torch.nn.functional.pad(order, (0, most - order.shape[2]))
    held = slot < count  # [B, 1, most]
    kept = torch.where(held, order[:, :, :most], 1 << 30).sort(-1).values
    b, h, i = torch.nonzero(held.expand(B, H, most), as_tuple=True)
    j = kept[b, h, i]
    src, dst = s["table"][b, j // page].long(), s["new_table"][b, i // page].long()
    for t in (*s["cache"], s["mass"]):
        t[dst, h, i % page] = t[src, h, j % page]
    s["kept"].copy_(torch.where(held, kept, -1))
    s["new_lens"].copy_(count.flatten())
    return {"new_lens": s["new_lens"], "kept": s["kept"], "mass": s["mass"], **_cache_out(s)}


def run(s):
    op, c = s["op"], s["case"]
    if own:
        from block_scaled_fp8_act_gb300 import fp8act
        if op == "rope":
            q = fp8act.fp8_rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["cache"],
                                       q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, axes=s["axes"],
                                       interleaved=c["interleaved"], q_out=s["out"])
            return {"q": q, **_cache_out(s)}
        if op == "evict":
            new_lens, kept = fp8act.fp8_kv_evict(s["cache"], s["mass"], s["table"], s["lens"], s["keep"], s["new_table"],
                                                 recent=c["recent"], first=c["first"], new_lens=s["new_lens"],
                                                 kept=s["kept"])
            return {"new_lens": new_lens, "kept": kept, "mass": s["mass"], **_cache_out(s)}
        how = {"soft_cap": c["cap"], "window": c["window"], "prefix_lens": s["prefix"], "first": s["first"],
               "slopes": s["slopes"]}
        if op == "attend":
            out = fp8act.fp8_kv_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu_q"], max_q_len=s["max_n"],
                                          out=s["out"], lse=s["lse"], **how)
            return {"out": out, "lse": s["lse"]}
        fp8act.fp8_kv_attention_mass(s["q"], s["cache"], s["table"], s["lens"], s["cu_q"], s["lse"], s["mass"],
                                     max_q_len=s["max_n"], accumulate=c["add"], **how)
        return s["mass"]
    return {"rope": _plain_rope, "attend": _plain_attend, "mass": _plain_mass, "evict": _plain_evict}[op](s)


# -------------------------------------------------------------------- work
def work(case):
    op, H, D = case["op"], case["H"], case["D"]
    if op == "rope":
        T, heads = case["T"], case["heads"]
        return {"bytes": T * (4 * heads * D + H * (4 * D + 2 * D + 8) + 8 * case["axes"] + 8) + 4 * case["rot"],
                "flops": T * (heads + H) * D * 8}
    B, L = case["B"], case["L"]
    low = min(case.get("n", 16), L)
    # the mean of lengths spread evenly over their logarithm, the first one the longest
    mean = (L - low) / math.log(L / low) if case["ragged"] and L > low else L
    total = L + (B - 1) * mean
    if op == "evict":
        kept = min(case["keep"], L) + (B - 1) * min(case["keep"], mean)
        return {"bytes": int(H * (4 * total + kept * (2 * (2 * D + 12) + 4))), "flops": int(H * total)}
    n, heads = case["n"], H * case["group"]

    def seen(length):  # positions that some new token sees, and the pairs of a sequence
        reach = min(length, case["window"] + n - 1 if case["window"] else length, case["doc"] + n - 1 if case["doc"] else length)
        prefix = min(case["prefix"], length - reach)
        each = max(reach - (n - 1) / 2, reach / 2)
        if case["window"]:
            each = min(each, case["window"])
        if case["doc"]:
            each = min(each, case["doc"])
        return reach + prefix, n * (each + prefix)

    (t0, p0), (t1, p1) = seen(L), seen(mean)
    tokens, pairs = t0 + (B - 1) * t1, p0 + (B - 1) * p1
    if op == "attend":
        return {"bytes": int(tokens * H * (2 * D + 8)) + B * n * heads * (4 * D + 4), "flops": int(4 * heads * D * pairs)}
    return {"bytes": int(tokens * H * (D + 4) + total * H * (8 if case["add"] else 4)) + B * n * heads * (2 * D + 4),
            "flops": int(2 * heads * D * pairs)}


# ----------------------------------------------------- definition, 64 bits
def _e4m3(x):
    """The nearest E4M3 value of a 64-bit one, ties to the even significand, saturating."""
    a = x.abs().clamp(max=E4M3_MAX)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3.0)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _exact_rope(s):
    case, page = s["case"], s["case"]["page"]
    half = case["rot"] // 2
    f = s["inv_freq"]
    angle = torch.stack([s["positions"][int(s["axes"][i]) if s["axes"] is not None else 0].double() * f[i] for i in range(half)], 1)
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    out = {}

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = weight.double() * x / torch.sqrt(torch.square(x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        at = torch.arange(half, device=DEV)
        i, j = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
        z = torch.complex(x[..., i], x[..., j]) * turn
        y = x.clone()
        y[..., i], y[..., j] = z.real, z.imag
        return y

    out["q"] = turned(s["q"], s["q_weight"])
    for name, x, codes, scales in (("k", turned(s["k"], s["k_weight"]), s["cache"][0], s["cache"][2]),
                                   ("v", s["v"].double(), s["cache"][1], s["cache"][3])):
        amax = x.abs().amax(-1, keepdim=True)
        scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
        values, new = codes.view(torch.float8_e4m3fn).double(), scales.double()
        values[s["slots"] // page, :, s["slots"] % page] = _e4m3(x / scale)
        new[s["slots"] // page, :, s["slots"] % page] = scale.squeeze(-1)
        out[name], out[name + "_scale"] = values, new
    return out


def _exact_rows(s):
    """For every sequence and KV head: its pages, the scores [n, group, L] and the cached values [L, D], in 64 bits."""
    c = s["case"]
    B, n, H, D, page, group = (c[k] for k in ("B", "n", "H", "D", "page", "group"))
    q = s["q"].double().view(B, n, H, group, D)
    for b in range(B):
        L = int(s["lens"][b])
        at = s["table"][b, :-(-L // page)].long()
        i, j = torch.arange(L - n, L, device=DEV).view(n, 1), torch.arange(L, device=DEV)
        hidden = j > i
        if c["window"]:
            hidden |= j <= i - c["window"]
        if s["first"] is not None:
            hidden |= j < s["first"][b * n:(b + 1) * n].view(n, 1)
        if s["prefix"] is not None:
            hidden &= j >= s["prefix"][b]
        for h in range(H):
            k, v = ((s["cache"][x][at, h].view(torch.float8_e4m3fn).double()
                     * s["cache"][x + 2][at, h].double().unsqueeze(-1)).flatten(0, 1)[:L] for x in (0, 1))
            x = torch.einsum("ngd,ld->ngl", q[b, :, h], k) / math.sqrt(D)
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if s["slopes"] is not None:
                x = x - torch.einsum("g,nl->ngl", s["slopes"].view(H, group)[h].double(), (i - j).abs().double())
            yield b, h, at, x.masked_fill(hidden.unsqueeze(1), -math.inf), v


def _exact_evict(s):
    c, page = s["case"], s["case"]["page"]
    names = {"k": 0, "v": 1, "k_scale": 2, "v_scale": 3}
    out = {x: (s["cache"][i].view(torch.float8_e4m3fn) if i < 2 else s["cache"][i]).double() for x, i in names.items()}
    out["mass"] = s["mass"].double()
    for b in range(c["B"]):
        L = int(s["lens"][b])
        count = min(L, c["keep"])
        recent = min(c["recent"], count)
        first = min(c["first"], count - recent)
        at = torch.arange(L, device=DEV)
        src = s["table"][b, at // page].long()
        for h in range(c["H"]):
            mass = s["mass"][src, h, at % page]
            rank = torch.argsort(mass[first:L - recent], descending=True, stable=True)[:count - recent - first] + first
            kept = torch.cat([at[:first], rank.sort().values, at[L - recent:]])
            dst = s["new_table"][b, at[:count] // page].long()
            for x in out.values():
                x[dst, h, at[:count] % page] = x[src[kept], h, kept % page]
    return {"new_lens": None, "kept": None, **out}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        return _exact_rope(s)
    if s["op"] == "evict":
        return _exact_evict(s)
    B, n, H, D, page, group = (case[k] for k in ("B", "n", "H", "D", "page", "group"))
    if s["op"] == "attend":
        out = torch.zeros((B, n, H, group, D), device=DEV, dtype=torch.float64)
        lse = torch.zeros((B, n, H, group), device=DEV, dtype=torch.float64)
        for b, h, _, x, v in _exact_rows(s):
            out[b, :, h] = torch.einsum("ngl,ld->ngd", torch.softmax(x, -1).nan_to_num(0.0), v)
            lse[b, :, h] = torch.logsumexp(x, -1)
        return {"out": out.view(B * n, -1, D), "lse": lse.view(B * n, -1)}
    mass, lse = s["mass"].double(), s["lse"].double().view(B, n, H, group, 1)
    for b, h, at, x, _ in _exact_rows(s):
        p = torch.where(x > -math.inf, torch.exp(x - lse[b, :, h]), 0.0).sum((0, 1))
        L = len(p)
        old = mass[at, h].flatten()
        if case["add"]:
            p[:L - n] += old[:L - n]
        mass[at, h] = torch.cat([p, old[L:]]).view(-1, page)
    return mass
