"""The operators around the cache as a serving loop uses them: a prompt with positions goes into the cache in chunks, its
last tokens say what matters, the rest is evicted, and decoding goes on over what stays. Every step is compared with the
definition in 64 bits on the codes that are in the cache, so that nothing but the step's own error is between them."""
from __future__ import annotations

import os
import sys

import pytest
import torch
from test_gpu_decoder_ops import check_attention, clean_status, fp8act, gen, randn  # noqa: F401  (fixtures too)
from test_gpu_kv_evict import reference as evict_ref
from test_gpu_rope_append import check_cached, rope_ref
from test_gpu_scores import cached, i32, scores_ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Loop:
    """Two sequences in one cache; `places` is a sequence's pages."""

    def __init__(self, fp8act, D, H, group, page, how, seed):  # noqa: F811
        self.f, self.D, self.H, self.group, self.page, self.how, self.seed = fp8act, D, H, group, page, how, seed
        self.cache = fp8act.kv_cache(60, H, page, D)
        self.mass = fp8act.kv_mass(self.cache)
        self.order = torch.randperm(60, device="cuda", generator=gen(seed)).to(torch.int32)
        self.inv = 1e4 ** (-2.0 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
        self.weights = [1 + 0.1 * randn(D, seed=seed + i) for i in (1, 2)]

    def step(self, table, before, n, pos0, seed, mass_rows, first):
        """n new tokens of every sequence at places `before` on and positions pos0 on; the last mass_rows add their weights."""
        f, B = self.f, len(before)
        T = B * n
        rows = randn(T, (self.group + 2) * self.H * self.D, seed=seed)
        q, k, v = (t.unflatten(1, (-1, self.D)) for t in rows.split([self.group * self.H * self.D] + 2 * [self.H * self.D], 1))
        at = (torch.tensor(before, device="cuda").unsqueeze(1) + torch.arange(n, device="cuda"))
        slots = (table.gather(1, at // self.page).long() * self.page + at % self.page).flatten()
        pos = (torch.tensor(pos0, device="cuda").unsqueeze(1) + torch.arange(n, device="cuda")).flatten()
        q = f.fp8_rope_append(q, k, v, pos, self.inv, slots, self.cache, q_weight=self.weights[0], k_weight=self.weights[1])
        lens = [b + n for b in before]
        cu, kv = i32([n * b for b in range(B + 1)]), i32(lens)
        lse = torch.empty(q.shape[:2], device="cuda")
        out = f.fp8_kv_attention(q, self.cache, table, kv, cu, max_q_len=n, lse=lse, **self.how)
        last = torch.cat([torch.arange(n * (b + 1) - mass_rows, n * (b + 1), device="cuda") for b in range(B)])
        f.fp8_kv_attention_mass(q[last], self.cache, table, kv, i32([mass_rows * b for b in range(B + 1)]), lse[last], self.mass,
                                max_q_len=mass_rows, accumulate=not first, old_lens=i32(before), **self.how)
        # the definition, on the cache as it is
        want, tol = rope_ref(rows[:, :self.group * self.H * self.D].unflatten(1, (-1, self.D)), self.weights[0], pos, self.inv, None, False)
        assert ((q.double() - want).abs() <= 2.0 ** -8 * want.abs() + tol).all()
        want, tol = rope_ref(k, self.weights[1], pos, self.inv, None, False)
        p, o = slots // self.page, slots % self.page
        check_cached(self.cache.k[p, :, o], self.cache.k_scale[p, :, o], want, tol)
        weights = []
        for rows_b, x, values in scores_ref(q, self.cache, table, lens, [n] * B, self.D ** -0.5, **self.how):
            w = torch.softmax(x, -1)
            ref, mag = (torch.einsum("nhl,lhd->nhd", w, t) for t in (values, values.abs()))
            check_attention(out[rows_b], ref, mag)
            weights.append(w[n - mass_rows:].unflatten(1, (self.H, self.group)).sum((0, 2)).T)  # [L, H]
        return lens, weights

    def masses(self, table, lens):
        return [self.mass[table[b, torch.arange(n, device="cuda") // self.page].long(), :, torch.arange(n, device="cuda") % self.page]
                for b, n in enumerate(lens)]


@pytest.mark.parametrize("D,H,group,page,how", [(128, 2, 6, 16, dict()), (128, 2, 6, 64, dict(soft_cap=20.0)),
                                                (64, 3, 4, 16, dict(soft_cap=30.0)), (256, 1, 2, 32, dict())])
def test_prompt_evict_decode(fp8act, D, H, group, page, how):  # noqa: F811
    loop = Loop(fp8act, D, H, group, page, how, seed=D + page)
    per = -(-160 // page)
    table = loop.order[:2 * per].view(2, per).contiguous()
    loop.mass.fill_(float("nan"))  # (pages that others had before)
    lens, w0 = loop.step(table, [0, 0], 90, [0, 0], 1, 16, True)
    total = [w.clone() for w in w0]
    lens, w1 = loop.step(table, lens, 60, lens, 2, 16, False)
    total = [torch.cat([t, torch.zeros_like(w[len(t):])]) + w for t, w in zip(total, w1)]
    for got, want in zip(loop.masses(table, lens), total):
        # (the new tokens' places start from zero; weights of 16 + 16 rows, each within 2^-12, lse's 2^-12 beside)
        assert ((got.double() - want).abs() <= 2.0 ** -10 * want + 1e-20).all()
    keep, fresh_pages = i32([40, 150]), -(-150 // page)
    fresh = loop.order[2 * per:2 * per + 2 * (fresh_pages + 1)].view(2, fresh_pages + 1).contiguous()
    want = evict_ref(loop.cache, loop.mass, table, i32(lens), keep, fresh, 10, 4)
    new_lens, kept = fp8act.fp8_kv_evict(loop.cache, loop.mass, table, i32(lens), keep, fresh, recent=10, first=4)
    assert torch.equal(new_lens.cpu(), want[0]) and torch.equal(kept.cpu(), want[1])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*loop.cache, loop.mass), want[2]))
    # decoding goes on at the places behind what stayed, at the positions that follow the whole prompt
    at, pos = new_lens.tolist(), list(lens)
    before = [m[:n].clone() for m, n in zip(loop.masses(fresh, at), at)]
    for i in range(3):
        at, w = loop.step(fresh, at, 1, pos, 10 + i, 1, False)
        pos = [p + 1 for p in pos]
        before = [torch.cat([b, torch.zeros_like(x[len(b):])]) + x for b, x in zip([b.double() for b in before], w)]
    for got, want in zip(loop.masses(fresh, at), before):
        assert ((got.double() - want).abs() <= 2.0 ** -10 * want + 1e-20).all()
    k, _ = cached(loop.cache, fresh, 0, at[0])
    assert torch.isfinite(k).all()


@pytest.mark.parametrize("kw", [dict(rope_theta=1e4), dict(rope_theta=1e6, soft_cap=8.0, window=50, head_dim=128, heads=12, kv_heads=2,
                                                           drafts=7, context=300, batch=2, page=64)])
def test_verify_step_with_positions(kw):
    """The example's step: its graph gives the eager step's results, and positions and the score function have a say."""
    import verify_step as ex
    from block_scaled_fp8_act_gb300 import fp8act as f
    f.load(build=True)
    c = ex.Config(**kw)
    d = ex.Decoder(c)
    state = ex.inputs(c, 1)
    want = d.step(*state)
    assert torch.isfinite(want[3]).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = d.step(*state)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    d.positions += 1000  # the new tokens move away from the cached ones
    assert not torch.equal(d.step(*state)[3], want[3])
    assert f.check_status() == 0


def test_past_four_gigabytes(fp8act):  # noqa: F811
    """Codes beyond 2^32 bytes: turned keys go there, are attended to, weighed and moved from one end to the other."""
    H, page, D = 8, 256, 256
    pages = (1 << 32) // (H * page * D) + 3
    cache = fp8act.kv_cache(pages, H, page, D)
    assert cache.k.numel() > 1 << 32
    mass = fp8act.kv_mass(cache)
    q, k, v = randn(5, 2 * H, D, seed=1), randn(5, H, D, seed=2), randn(5, H, D, seed=3)
    inv = 1e4 ** (-2.0 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
    pos = torch.arange(5, device="cuda")
    at = (pages - 1) * page + pos
    turned = fp8act.fp8_rope_append(q, k, v, pos, inv, at, cache)
    want, tol = rope_ref(k, None, pos, inv, None, False)
    check_cached(cache.k[pages - 1, :, :5].transpose(0, 1), cache.k_scale[pages - 1, :, :5].T, want, tol)
    table, cu = i32([[pages - 1]]), i32([0, 5])
    lse = torch.empty((5, 2 * H), device="cuda")
    out = fp8act.fp8_kv_attention(turned, cache, table, i32([5]), cu, max_q_len=5, lse=lse, window=3, soft_cap=10.0)
    fp8act.fp8_kv_attention_mass(turned, cache, table, i32([5]), cu, lse, mass, max_q_len=5, accumulate=False, window=3, soft_cap=10.0)
    for rows, x, values in scores_ref(turned, cache, table, [5], [5], D ** -0.5, window=3, soft_cap=10.0):
        p = torch.softmax(x, -1)
        check_attention(out[rows], *(torch.einsum("nhl,lhd->nhd", p, t) for t in (values, values.abs())))
        got = mass[pages - 1, :, :5].T.double()
        w = p.unflatten(1, (H, 2)).sum((0, 2)).T
        assert ((got - w).abs() <= 2.0 ** -11 * w + 1e-20).all()
    new_lens, kept = fp8act.fp8_kv_evict(cache, mass, table, i32([5]), i32([4]), i32([[pages - 2]]), recent=2)
    for h in range(H):
        assert torch.equal(cache.k[pages - 2, h, :4], cache.k[pages - 1, h, kept[0, h, :4].long()])
    assert new_lens.tolist() == [4] and (kept[0, :, 2:4].cpu() == torch.tensor([3, 4])).all()
