"""GPU tests of attention with capped and biased scores, windows, prefixes and documents, and of the weights that
cached tokens get, against the definitions in 64 bits on the same inputs.

Tolerances, from the arithmetic. Outputs as for plain attention (test_gpu_decoder_ops.py), |error| <= 2^-8 |o| + 2^-10
sum p |v|: a cap is off by 2^-21 of itself and a bias by 2^-23, for caps of at most 100 and biases that leave a weight
above 2^-24 (at most 17) far below the 2^-13 that the product's own error is bounded by. The log-sum-exp is off by the
scores' 2^-13 and its own roundings. A weight exp(x - lse) is off by x's 2^-13 and the exponential's and the sum's
roundings, 2^-20 with at most 8000 rows: mass is within 2^-12 of itself, plus what lies below the smallest exponent.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch
from test_gpu_decoder_ops import (INDEX, attend, check_attention, clean_status, fp8act, gen, make_cache,  # noqa: F401
                                  randn)

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cached(cache, table, b, L):
    """fp64 keys and values [L, H, D] of a sequence."""
    at = table[b, :-(-L // cache.k.shape[2])].long()
    return [(c[at].view(torch.float8_e4m3fn).double() * s[at].double().unsqueeze(-1)).transpose(1, 2).flatten(0, 1)[:L]
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


def scores_ref(q, cache, table, lens, ns, scale, soft_cap=0.0, window=0, prefix_lens=None, first=None, slopes=None):
    """Per sequence: (its rows of q, scores fp64 [n, Hq, L] with -inf where nothing is seen, values)."""
    Hq, H = q.shape[1], cache.k.shape[1]
    t0 = 0
    for b, (L, n) in enumerate(zip(lens, ns)):
        rows = slice(t0, t0 + n)
        t0 += n
        k, v = (t.repeat_interleave(Hq // H, 1) for t in cached(cache, table, b, L))
        x = torch.einsum("nhd,lhd->nhl", q[rows].double(), k) * scale
        if soft_cap:
            x = soft_cap * torch.tanh(x / soft_cap)
        i, j = torch.arange(L - n, L, device="cuda").view(n, 1), torch.arange(L, device="cuda")
        if slopes is not None:
            x = x - slopes.double().view(1, Hq, 1) * (i - j).abs().unsqueeze(1)
        seen = j <= i
        if window:
            seen = seen & (j > i - window)
        if first is not None:
            seen = seen & (j >= first[rows].view(n, 1))
        if prefix_lens is not None:
            seen = seen | (j < int(prefix_lens[b]))
        yield rows, x.masked_fill(~seen.unsqueeze(1), -math.inf), v


def check(fp8act, q, cache, table, lens, ns, softmax_scale=None, **how):  # noqa: F811
    """Attention, its lse, and the masses of both kinds of call."""
    scale = softmax_scale or q.shape[2] ** -0.5
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = attend(fp8act, q, cache, table, lens, ns, lse=lse, softmax_scale=softmax_scale, **how)
    H, page = cache.k.shape[1:3]
    group = q.shape[1] // H
    ref, mag, lref = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros_like(q, dtype=torch.float64), []
    masses = []
    for rows, x, v in scores_ref(q, cache, table, lens, ns, scale, **{k: w for k, w in how.items() if k != "max_q_len"}):
        p = torch.softmax(x, -1).nan_to_num(0.0)
        ref[rows] = torch.einsum("nhl,lhd->nhd", p, v)
        mag[rows] = torch.einsum("nhl,lhd->nhd", p, v.abs())
        lref.append(torch.logsumexp(x, -1) if x.shape[2] else torch.full(x.shape[:2], -math.inf, device="cuda", dtype=torch.float64))
        shift = torch.where(lse[rows] == -math.inf, 0.0, lse[rows].double()).unsqueeze(-1)
        masses.append(torch.exp(x - shift).unflatten(1, (H, group)).sum((0, 2)).T)  # [L, H]
    check_attention(out, ref, mag)
    lref = torch.cat(lref)
    empty = lref == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (out[empty] == 0).all()
    assert ((lse.double() - lref)[~empty].abs() <= 2.0 ** -12 + 2.0 ** -20 * lref[~empty].abs()).all()

    cu, kv = i32(np.concatenate([[0], np.cumsum(ns)])), i32(lens)
    old = torch.rand((len(cache.k), H, page), device="cuda", generator=gen(1))
    for accumulate in (True, False):
        mass = old.clone()
        # what the new tokens' places hold is not read
        for b, (L, n) in enumerate(zip(lens, ns)):
            at = torch.arange(max(L - n, 0) if accumulate else 0, L, device="cuda")
            mass[table[b, at // page].long(), :, at % page] = math.nan
        want = mass.double()
        tol = torch.zeros_like(want)
        for b, (L, n) in enumerate(zip(lens, ns)):
            at = torch.arange(L, device="cuda")
            p, o = table[b, at // page].long(), at % page
            base = torch.where((at < L - n).unsqueeze(1) & accumulate, want[p, :, o], 0.0)
            want[p, :, o] = base + masses[b]
            tol[p, :, o] = 2.0 ** -12 * masses[b] + 2.0 ** -22 * want[p, :, o] + 1e-30
        args = (q, cache, table, kv, cu, lse, mass)
        how.setdefault("max_q_len", max(ns))
        fp8act.fp8_kv_attention_mass(*args, softmax_scale=softmax_scale, accumulate=accumulate, **how)
        same = mass.double() == want
        assert torch.equal(torch.isnan(mass), torch.isnan(want))
        assert (same | torch.isnan(want) | ((mass.double() - want).abs() <= tol)).all()
    return out, lse


def options(lens, ns, Hq, seed):
    """Score functions to go through: each alone, and together."""
    rng = np.random.default_rng(seed)
    firsts = []
    for L, n in zip(lens, ns):  # not falling; some before the cache and some behind the token
        firsts += sorted(int(x) for x in rng.integers(-2, L + 3, n))
    prefix = [int(rng.integers(-1, L + 5)) for L in lens]
    slopes = torch.tensor(2.0 ** (-8 * (np.arange(Hq) + 1) / Hq), dtype=torch.float32, device="cuda")
    most = max(lens)
    return {"cap": dict(soft_cap=20.0), "window 1": dict(window=1), "window": dict(window=max(1, most // 3)),
            "wide window": dict(window=2 ** 31 - 1), "prefix": dict(prefix_lens=i32(prefix)), "documents": dict(first=i32(firsts)),
            "bias": dict(slopes=slopes), "sinks": dict(window=max(1, most // 4), prefix_lens=i32([min(4, L) for L in lens])),
            "all": dict(soft_cap=5.0, window=max(2, most // 2), prefix_lens=i32([p // 3 for p in prefix]), first=i32(firsts),
                        slopes=-slopes)}


KINDS = ["cap", "window 1", "window", "wide window", "prefix", "documents", "bias", "sinks", "all"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,group,n", [(64, 1, 1), (64, 6, 3), (64, 8, 20), (128, 6, 1), (128, 3, 2), (128, 6, 3), (128, 6, 8),
                                       (128, 6, 9), (128, 5, 40), (256, 2, 1), (256, 4, 3), (256, 8, 8)])
def test_scores_and_masses(fp8act, kind, D, group, n):  # noqa: F811
    H, page = 2, 16
    lens = [n, 63 + n, 64, 65, 130, 1000, 1]
    ns = [min(n, L) if b % 2 else n for b, L in enumerate(lens)]  # some with more new tokens than cached
    ns = [min(m, L) if kind in ("documents", "all") else m for m, L in zip(ns, lens)]
    cache, table = make_cache(fp8act, lens, H, D, page, seed=D + group)
    q = randn(sum(ns), H * group, D, seed=3)
    check(fp8act, q, cache, table, lens, ns, **options(lens, ns, H * group, D + n)[kind])


@pytest.mark.parametrize("kind", ["cap", "window", "documents", "sinks", "all"])
@pytest.mark.parametrize("n", [1, 8, 30])
def test_scores_over_long_contexts(fp8act, kind, n):  # noqa: F811
    lens, ns = [9000, 3000], [n, n]
    cache, table = make_cache(fp8act, lens, 2, 128, 64, seed=n)
    q = randn(2 * n, 12, 128, seed=n)
    how = options(lens, ns, 12, n)[kind]
    first = check(fp8act, q, cache, table, lens, ns, **how)
    again = check(fp8act, q, cache, table, lens, ns, **how)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_prompt_whose_tokens_are_all_new(fp8act, D):  # noqa: F811
    """Several row tiles, each with its own part of the cache; a bidirectional prefix; more rows than are staged at once."""
    lens = ns = [333, 64, 150]
    cache, table = make_cache(fp8act, lens, 1, D, 16, seed=D)
    q = randn(sum(ns), 6, D, seed=4)
    for kind, how in options(lens, ns, 6, 5).items():
        check(fp8act, q, cache, table, lens, ns, **how)
    check(fp8act, q, cache, table, lens, ns, prefix_lens=i32([333, 10, 70]), window=20)


def test_the_hint_changes_nothing_but_the_tiles(fp8act):  # noqa: F811
    lens, ns = [700, 90], [40, 33]
    cache, table = make_cache(fp8act, lens, 2, 128, 32, seed=9)
    q = randn(73, 8, 128, seed=10)
    how = options(lens, ns, 8, 11)["all"]
    for hint in (1, 3, 12, 100):
        check(fp8act, q, cache, table, lens, ns, max_q_len=hint, **how)


def test_neutral_scores_are_plain_attention(fp8act):  # noqa: F811
    """A window over everything, no prefix, documents that start at 0: the plain call's results."""
    for n, D in ((1, 128), (8, 64), (20, 128), (3, 256)):
        lens, ns = [500, 33], [n, n]
        cache, table = make_cache(fp8act, lens, 2, D, 16, seed=n)
        q = randn(2 * n, 8, D, seed=n)
        lse = torch.empty((2 * n, 8), device="cuda"), torch.empty((2 * n, 8), device="cuda")
        plain = attend(fp8act, q, cache, table, lens, ns, lse=lse[0])
        for how in (dict(), dict(soft_cap=0.0, window=0), dict(soft_cap=None, window=None)):
            assert torch.equal(attend(fp8act, q, cache, table, lens, ns, lse=lse[1], **how), plain) and torch.equal(*lse)
        got = attend(fp8act, q, cache, table, lens, ns, lse=lse[1], prefix_lens=i32([0, 0]), first=i32([0] * 2 * n), window=600)
        ref = plain.double()
        assert ((got.double() - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -9 * ref.abs().amax(-1, keepdim=True)).all()
        assert ((lse[0] - lse[1]).abs() <= 2.0 ** -12).all()


@pytest.mark.parametrize("cap", [0.5, 30.0, 1e30, 1e-30])
@pytest.mark.parametrize("n", [2, 30])
def test_caps_of_large_scores(fp8act, cap, n):  # noqa: F811
    """Scores of +-100 times a scale of up to 100: far into the cap's flat ends, and caps that leave nothing or all."""
    lens, ns = [600, 50], [n, n]
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=13)
    q = randn(2 * n, 8, 128, seed=14)
    for scale in ((1.0, 100.0) if cap <= 30 else (1.0,)):
        lse = torch.empty((2 * n, 8), device="cuda")
        out = attend(fp8act, q, cache, table, lens, ns, soft_cap=cap, softmax_scale=scale, lse=lse)
        for rows, x, v in scores_ref(q, cache, table, lens, ns, scale, soft_cap=cap):
            p = torch.softmax(x, -1)
            ref, mag = (torch.einsum("nhl,lhd->nhd", p, w) for w in (v, v.abs()))
            check_attention(out[rows], ref, mag)
            # (a score of 100 has an fp32 error of up to 2^-13 before the cap)
            assert ((lse[rows].double() - torch.logsumexp(x, -1)).abs() <= 2.0 ** -12 + 2.0 ** -20 * lse[rows].abs()).all()


@pytest.mark.parametrize("n", [1, 8, 30])
def test_poisoned_tokens_reach_who_sees_them(fp8act, n):  # noqa: F811
    """A NaN scale inside a window or a prefix poisons the rows that see it; outside of both it does nothing."""
    lens, ns = [400], [n]
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=15)
    q = randn(n, 12, 128, seed=16)
    how = dict(window=50, prefix_lens=i32([20]))
    clean, lse = check(fp8act, q, cache, table, lens, ns, **how)
    for pos, hits in ((200, False), (30, False), (10, True), (400 - n - 5, True)):
        page, off = int(table[0, pos // 16]), pos % 16
        for name in ("k_scale", "v_scale"):
            bad = fp8act.KvCache(*(t.clone() for t in cache))
            getattr(bad, name)[page, 1, off] = math.nan
            out = attend(fp8act, q, bad, table, lens, ns, **how)
            assert torch.equal(out[:, :6], clean[:, :6])
            assert torch.isnan(out[:, 6:]).all() if hits else torch.equal(out, clean)
        mass = torch.zeros(cache.k_scale.shape, device="cuda")
        poisoned = fp8act.KvCache(*(t.clone() for t in cache))
        poisoned.k_scale[page, 1, off] = math.nan
        fp8act.fp8_kv_attention_mass(q, poisoned, table, i32(lens), i32([0, n]), lse, mass, **how)
        bad = torch.isnan(mass)
        assert bad.sum() == (1 if hits else 0) and bool(bad[page, 1, off]) == hits


def test_unseen_positions_are_not_read(fp8act):  # noqa: F811
    """Pages that no row sees may be out of range; they would be reported if the table were followed."""
    lens, ns = [5000], [1]
    cache, table = make_cache(fp8act, lens, 1, 128, 16, seed=17)
    q = randn(1, 6, 128, seed=18)
    want = attend(fp8act, q, cache, table, lens, ns, window=64, prefix_lens=i32([32]))
    cut = table.clone()
    cut[0, 16:300] = -1
    assert torch.equal(attend(fp8act, q, cache, cut, lens, ns, window=64, prefix_lens=i32([32])), want)
    assert fp8act.check_status() == 0
    attend(fp8act, q, cache, cut, lens, ns, window=4000)
    assert fp8act.check_status() == INDEX


def test_documents_that_fall_are_reported(fp8act):  # noqa: F811
    for n in (3, 30):
        lens, ns = [200, 90], [n, n]
        cache, table = make_cache(fp8act, lens, 1, 128, 16, seed=19)
        q = randn(2 * n, 4, 128, seed=20)
        lse = torch.empty((2 * n, 4), device="cuda")
        fine = [5] * (n - 1) + [80] + [2] * n  # (falls between the sequences, not in one)
        attend(fp8act, q, cache, table, lens, ns, first=i32(fine), lse=lse)
        assert fp8act.check_status() == 0
        bad = fine[:-2] + [9, 3]
        attend(fp8act, q, cache, table, lens, ns, first=i32(bad))
        assert fp8act.check_status() == INDEX
        fp8act.fp8_kv_attention_mass(q, cache, table, i32(lens), i32([0, n, 2 * n]), lse, torch.zeros_like(cache.k_scale),
                                     first=i32(bad))
        assert fp8act.check_status() == INDEX


def test_mass_rows_of_no_sequence_and_empty_sequences(fp8act):  # noqa: F811
    """Sequences without new tokens keep their weights, or lose them if those are replaced; NaN rows past the last one."""
    lens, ns = [100, 50, 0, 70], [2, 0, 0, 1]
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=21)
    q = randn(5, 4, 128, seed=22)
    q[3:] = math.nan
    lse = torch.full((5, 4), math.nan, device="cuda")
    cu, kv = i32([0, 2, 2, 2, 3]), i32(lens)
    fp8act.fp8_kv_attention(q, cache, table, kv, cu, lse=lse)
    old = torch.rand(cache.k_scale.shape, device="cuda", generator=gen(2))
    for accumulate in (True, False):
        mass = old.clone()
        fp8act.fp8_kv_attention_mass(q, cache, table, kv, cu, lse, mass, accumulate=accumulate)
        assert torch.isfinite(mass).all()
        at = torch.arange(50, device="cuda")
        mine = mass[table[1, at // 16].long(), :, at % 16]
        assert torch.equal(mine, old[table[1, at // 16].long(), :, at % 16]) if accumulate else (mine == 0).all()
        assert torch.equal(mass[table[0, 6].long(), :, 4:], old[table[0, 6].long(), :, 4:])  # past its 100 tokens
    # all rows' weights sum to 1 a row
    total = sum(mass[table[b, torch.arange(L, device="cuda") // 16].long(), :, torch.arange(L, device="cuda") % 16].sum()
                for b, L in enumerate(lens))
    assert abs(float(total) - 12) < 12 * 2.0 ** -11


def test_mass_streams_and_graphs(fp8act):  # noqa: F811
    lens, ns = [3000, 200], [8, 8]
    cache, table = make_cache(fp8act, lens, 2, 128, 64, seed=23)
    q = randn(16, 12, 128, seed=24)
    how = dict(soft_cap=30.0, window=500)
    out, lse = check(fp8act, q, cache, table, lens, ns, **how)
    args = (q, cache, table, i32(lens), i32([0, 8, 16]), lse)
    want = torch.zeros(cache.k_scale.shape, device="cuda")
    fp8act.fp8_kv_attention_mass(*args, want, **how)
    side = torch.cuda.Stream()
    got = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    fp8act.fp8_kv_attention_mass(*args, got, stream=side, **how)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    with torch.cuda.graph(graph):
        fp8act.fp8_kv_attention(*args[:5], out=again, lse=lse2, max_q_len=8, **how)
        fp8act.fp8_kv_attention_mass(*args[:5], lse2, got, accumulate=False, **how)
    for _ in range(2):
        got.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        there = torch.zeros_like(want, dtype=torch.bool)
        for b, L in enumerate(lens):
            at = torch.arange(L, device="cuda")
            there[table[b, at // 64].long(), :, at % 64] = True
        assert torch.equal(again, out) and torch.equal(got[there], want[there]) and (got[~there] == 3).all()


def test_score_refusals(fp8act):  # noqa: F811
    lens, ns = [100], [2]
    cache, table = make_cache(fp8act, lens, 2, 64, 16, seed=25)
    q = randn(2, 4, 64, seed=26)
    mass, lse = torch.zeros(cache.k_scale.shape, device="cuda"), torch.zeros((2, 4), device="cuda")
    kv, cu = i32(lens), i32([0, 2])

    def both(**how):
        yield lambda: fp8act.fp8_kv_attention(q, cache, table, kv, cu, **how)
        yield lambda: fp8act.fp8_kv_attention_mass(q, cache, table, kv, cu, lse, mass, **how)
    for how in (dict(soft_cap=-1.0), dict(soft_cap=math.nan), dict(soft_cap=math.inf), dict(soft_cap=1e-35), dict(window=-1)):
        for call in both(**how):
            with pytest.raises(fp8act.Fp8ActError):
                call()
    for how in (dict(prefix_lens=torch.zeros(1, device="cuda")), dict(first=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(slopes=torch.zeros(4, dtype=torch.float64, device="cuda")), dict(slopes=torch.zeros(4))):
        for call in both(**how):
            with pytest.raises(TypeError):
                call()
    for how in (dict(prefix_lens=i32([0, 0])), dict(first=i32([0])), dict(slopes=torch.zeros(2, device="cuda")), dict(window=1 << 40)):
        for call in both(**how):
            with pytest.raises(ValueError):
                call()
    for bad in (dict(lse=lse[:1]), dict(mass=mass[:1]), dict(lse=lse.double()), dict(mass=mass.half())):
        a = dict(lse=lse, mass=mass)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            fp8act.fp8_kv_attention_mass(q, cache, table, kv, cu, **a)


@pytest.mark.parametrize("n,group", [(6, 6), (9, 6), (16, 6), (32, 6), (43, 6), (64, 4), (100, 7)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_masses_of_many_rows(fp8act, n, group, page):  # noqa: F811
    """The tcgen05 kernel of head size 128: one to three times its rows, ragged tiles of 128 tokens, pages of every size."""
    lens = [n, 127, 128, 129, 1, 700, 0, 2500]
    ns = [min(n, L) if b % 2 == 0 else n for b, L in enumerate(lens)]
    cache, table = make_cache(fp8act, lens, 2, 128, page, seed=n + page)
    q = randn(sum(ns), 2 * group, 128, seed=3)
    check(fp8act, q, cache, table, lens, ns)
    check(fp8act, q, cache, table, lens, ns, **options(lens, ns, 2 * group, n)["sinks"])


def test_masses_of_many_rows_over_long_contexts(fp8act):  # noqa: F811
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(1, 3000, 30)] + [40000]
    ns = [min(int(x), L) for x, L in zip(rng.integers(0, 40, 31), lens)]
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=63)
    q = randn(sum(ns), 8, 128, seed=64)
    for hint in (20, 100):
        check(fp8act, q, cache, table, lens, ns, max_q_len=hint)


def test_mass_wait_that_runs_out(fp8act):  # noqa: F811
    """The tcgen05 kernel leaves cleanly when a copy never comes, and the next call is right."""
    lens, ns = [3000, 100], [16, 16]
    cache, table = make_cache(fp8act, lens, 2, 128, 64, seed=71)
    q = randn(32, 12, 128, seed=72)
    _, lse = check(fp8act, q, cache, table, lens, ns)
    args = (q, cache, table, i32(lens), i32([0, 16, 32]), lse)
    mass = torch.zeros(cache.k_scale.shape, device="cuda")
    try:
        fp8act.set_wait_limit(1_000_000, True)
        fp8act.fp8_kv_attention_mass(*args, mass, max_q_len=16)
        assert fp8act.check_status() == 5  # FP8ACT_ERR_TIMEOUT
    finally:
        fp8act.set_wait_limit(-1, False)
    check(fp8act, q, cache, table, lens, ns)


@pytest.mark.parametrize("n", [2, 30])
def test_mass_of_the_last_tokens_of_a_chunk(fp8act, n):  # noqa: F811
    """With old_lens, places that hold a token's first weight start from zero whether the token is passed or not."""
    lens, ns, old = [700, 300, 40, 90], [n, n, 0, n], [600, 0, 25, 200]
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=81)
    q = randn(sum(ns), 12, 128, seed=82)
    lse = torch.empty(q.shape[:2], device="cuda")
    attend(fp8act, q, cache, table, lens, ns, lse=lse)
    args = (q, cache, table, i32(lens), i32(np.concatenate([[0], np.cumsum(ns)])), lse)
    before = torch.rand(cache.k_scale.shape, device="cuda", generator=gen(3))
    alone = torch.zeros_like(before)
    fp8act.fp8_kv_attention_mass(*args, alone, max_q_len=n, accumulate=False)
    mass = before.clone()
    for b, (L, o) in enumerate(zip(lens, old)):
        at = torch.arange(min(o, L), L, device="cuda")
        mass[table[b, at // 16].long(), :, at % 16] = math.nan
    fp8act.fp8_kv_attention_mass(*args, mass, max_q_len=n, old_lens=i32(old))
    for b, (L, o) in enumerate(zip(lens, old)):
        at = torch.arange(L, device="cuda")
        p, s = table[b, at // 16].long(), at % 16
        want = torch.where((at < o).unsqueeze(1), before[p, :, s], 0.0) + alone[p, :, s]
        # (with more rows than one pass takes the old weight is added to the first pass's sum and the second's to that: each of
        # the two sides rounds at most twice, 2^-24 of a sum that only grows)
        assert ((mass[p, :, s].double() - want.double()).abs() <= 2.0 ** -22 * want).all()
