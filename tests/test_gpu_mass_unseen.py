"""GPU tests of the weights of cached tokens where a window or a document has left pages behind: entries of the page table
that no new token sees and whose weights stay are not followed, whatever stands there.

Tolerances as in test_gpu_scores.py: a weight is within 2^-12 of itself, and adding it to one that was there rounds once.
"""
from __future__ import annotations

import math

import pytest
import torch
from test_gpu_decoder_ops import attend, clean_status, fp8act, gen, make_cache, randn  # noqa: F401  (fixtures too)
from test_gpu_scores import i32, scores_ref

pytestmark = pytest.mark.gpu

LENS, OLD = [2000, 900, 300], [1950, 880, 300]


def scores(kind, ns):
    """(Score function, positions from which on a sequence's rows see everything that they see behind its prefix.)"""
    if kind == "window":
        return dict(window=200), [L - n - 199 for L, n in zip(LENS, ns)]
    if kind == "sinks":
        return dict(window=77, prefix_lens=i32([4, 40, 0])), [L - n - 76 for L, n in zip(LENS, ns)]
    starts = [1111, 703, 255]
    return dict(first=i32([s for s, n in zip(starts, ns) for _ in range(n)])), starts


@pytest.mark.parametrize("kind", ["window", "sinks", "documents"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n", [1, 8, 30])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_unseen_pages_are_neither_read_nor_written(fp8act, D, n, page, kind):  # noqa: F811
    H, group, ns = 2, 6, [n] * 3
    cache, table = make_cache(fp8act, LENS, H, D, page, seed=D + n)
    q = randn(3 * n, H * group, D, seed=n)
    how, start = scores(kind, ns)
    lse = torch.empty(q.shape[:2], device="cuda")
    attend(fp8act, q, cache, table, LENS, ns, lse=lse, **how)
    prefix = how["prefix_lens"].tolist() if "prefix_lens" in how else [0, 0, 0]
    before = torch.rand(cache.k_scale.shape, device="cuda", generator=gen(n))

    def weights(entries, old, calls=1):
        mass = before.clone()
        for _ in range(calls):
            fp8act.fp8_kv_attention_mass(q, cache, entries, i32(LENS), i32([0, n, 2 * n, 3 * n]), lse, mass, max_q_len=n,
                                         old_lens=old, **how)
        return mass

    for old in (None, i32(OLD)):
        kept = [L - n for L in LENS] if old is None else OLD
        full = weights(table, old)
        for b, (rows, x, _) in enumerate(scores_ref(q, cache, table, LENS, ns, D ** -0.5, **how)):
            w = torch.exp(x - lse[rows].double().unsqueeze(-1)).unflatten(1, (H, group)).sum((0, 2)).T
            at = torch.arange(LENS[b], device="cuda")
            p, o = table[b, at // page].long(), at % page
            want = torch.where((at < kept[b]).unsqueeze(1), before[p, :, o].double(), 0.0) + w
            assert ((full[p, :, o].double() - want).abs() <= 2.0 ** -12 * w + 2.0 ** -22 * want + 1e-30).all()
        # pages that were given back: nobody's, or another sequence's that gets weight in the same call
        unseen = [[i for i in range(-(-prefix[b] // page), min(start[b], kept[b]) // page)] for b in range(3)]
        assert len(unseen[0]) > 5 and len(unseen[1]) > 5
        nobody, other = table.clone(), table.clone()
        last = [(L - 1) // page for L in LENS]
        for b in range(3):
            nobody[b, unseen[b]] = -1
            to = (b + 1) % 3
            for k, i in enumerate(unseen[b]):
                other[b, i] = table[to, last[to] - k % (max(last[to] - start[to] // page, 0) + 1)]
        nobody[2, unseen[2][:1]] = 1 << 30
        for entries in (nobody, other):
            assert torch.equal(weights(entries, old), full)
            assert fp8act.check_status() == 0
        assert torch.equal(weights(other, old, 20), weights(table, old, 20))


@pytest.mark.parametrize("n", [1, 8, 30])
def test_sequences_without_new_tokens_beside_windows(fp8act, n):  # noqa: F811
    """No new tokens: nothing is seen, a prefix neither, and only places from old_lens on are written."""
    lens, ns = [700, 500, 600], [n, 0, n]
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=n)
    q = randn(2 * n, 12, 128, seed=n)
    how = dict(window=100, prefix_lens=i32([0, 30, 5]))
    lse = torch.empty(q.shape[:2], device="cuda")
    attend(fp8act, q, cache, table, lens, ns, lse=lse, **how)
    args = (i32(lens), i32([0, n, n, 2 * n]), lse)
    table[1, :20] = -1
    mass = torch.full(cache.k_scale.shape, math.nan, device="cuda")
    fp8act.fp8_kv_attention_mass(q, cache, table, *args, mass, max_q_len=n, **how)
    written = ~torch.isnan(mass[table[1, 20:].clamp(min=0).long()])
    assert not written.any()
    fp8act.fp8_kv_attention_mass(q, cache, table, *args, mass, max_q_len=n, old_lens=i32([700 - n, 330, 600 - n]), **how)
    at = torch.arange(320, 500, device="cuda")
    got = mass[table[1, at // 16].long(), :, at % 16]
    assert torch.isnan(got[:10]).all() and (got[10:] == 0).all()
    assert fp8act.check_status() == 0
