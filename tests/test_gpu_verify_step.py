"""The example's draft-verify step against the same step in plain fp32 / fp64 torch.

Both sides quantise the same weights and round to bf16 and E4M3 at the same
places, so they differ where a value near a rounding boundary falls to the
other side: a bf16 result by one unit, an E4M3 code by one step of 2^-3 of its
value at most. With every code of every activation off by half a step (2^-4)
the logits' relative L2 error would be 2^-4; that is the bound.
"""
from __future__ import annotations

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def dequant(w, sw):
    n, k = w.shape
    return w.view(torch.float8_e4m3fn).double() * sw.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)


def quant(y):
    g = y.float().unflatten(-1, (-1, 128))
    amax = g.abs().amax(-1, keepdim=True)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    return ((g / s).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s.double()).flatten(-2)


def norm(h, w):
    return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w.double()


def heads_quant(x):
    s = x.float().abs().amax(-1, keepdim=True) / 448.0
    return (x.float() / s).to(torch.float8_e4m3fn).double() * s.double()


def reference(d, tokens):
    c, n, width = d.c, tokens.shape[1], d.c.heads * d.c.head_dim
    x = d.embed[tokens.reshape(-1)].double()
    residual = None
    for w, cache in zip(d.layers, d.caches):
        h = x if residual is None else x + residual
        residual = h.bfloat16().double()
        qkv = (quant(norm(h, w["norm1"])) @ dequant(*w["qkv"]).T).bfloat16()
        q = qkv[:, :width].double().unflatten(1, (c.heads, c.head_dim)).unflatten(0, (c.batch, n))
        new = [heads_quant(t.unflatten(1, (c.kv_heads, c.head_dim))).unflatten(0, (c.batch, n))
               for t in qkv[:, width:].split(d.kv_width, 1)]
        at = d.table.long()
        old = [(codes[at].view(torch.float8_e4m3fn).double() * s[at].double().unsqueeze(-1))
               .transpose(2, 3).flatten(1, 2)[:, :c.context] for codes, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
        k, v = (torch.cat([o, m], 1).repeat_interleave(c.heads // c.kv_heads, 2) for o, m in zip(old, new))
        x = torch.einsum("bnhd,blhd->bhnl", q, k) * c.head_dim ** -0.5
        hidden = torch.arange(c.context + n, device="cuda") > c.context + torch.arange(n, device="cuda").unsqueeze(1)
        p = torch.softmax(x.masked_fill(hidden, -torch.inf), -1)
        o = torch.einsum("bhnl,blhd->bnhd", p, v).reshape(c.batch * n, width).bfloat16()
        x = (quant(o) @ dequant(*w["out"]).T).bfloat16().double()
        h = x + residual
        residual = h.bfloat16().double()
        gate, up = (quant(norm(h, w["norm2"])) @ dequant(*w["gate_up"]).T).bfloat16().double().chunk(2, -1)
        x = (quant(gate * torch.sigmoid(gate) * up) @ dequant(*w["down"]).T).bfloat16().double()
    return (quant(norm(x + residual, d.norm)) @ dequant(*d.head).T).unflatten(0, (c.batch, n))


@pytest.mark.parametrize("kw", [dict(), dict(head_dim=128, heads=12, kv_heads=2, drafts=7, context=300, batch=2, page=64),
                                dict(head_dim=128, heads=8, kv_heads=1, drafts=9, context=50, layers=1)])
def test_step(kw):
    import verify_step as ex
    from block_scaled_fp8_act_gb300 import fp8act
    fp8act.load(build=True)
    c = ex.Config(**kw)
    d = ex.Decoder(c)
    state = ex.inputs(c, 1)
    accepted, tokens, prob, logits = d.step(*state)
    want = reference(d, torch.cat([state[0].unsqueeze(1), state[1]], 1).long())
    assert (logits.double() - want).norm() <= 2.0 ** -4 * want.norm()
    from test_gpu_decoder_ops import check_verify
    again = check_verify(fp8act, logits, state[2], state[1], *state[3:])  # the verification of the step's own logits
    assert torch.equal(again[0], accepted) and torch.equal(again[1], tokens) and torch.equal(again[2], prob)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = d.step(*state)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (accepted, tokens, prob, logits)))
    assert fp8act.check_status() == 0
