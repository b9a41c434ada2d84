"""GPU tests of the eviction: which tokens stay is decided by comparisons and they are copied, so everything is exact."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch
from test_gpu_decoder_ops import INDEX, clean_status, fp8act, gen  # noqa: F401  (fixtures too)

pytestmark = pytest.mark.gpu


def problem(fp8act, lens, keep, H, D, page, seed, room=None, spare=2):  # noqa: F811
    """A cache of random bytes (the copy looks at none of them), weights, tables of old and new pages."""
    B = len(lens)
    per = max(1, -(-max(lens) // page))
    new = max(1, -(-max(keep) // page)) if room is None else room
    pages = B * (per + new) + spare
    g = gen(seed)
    codes = [torch.randint(0, 256, (pages, H, page, D), device="cuda", generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.rand((pages, H, page), device="cuda", generator=g) for _ in range(2)]
    cache = fp8act.KvCache(*codes, *scales)
    mass = torch.exp(3 * torch.randn((pages, H, page), device="cuda", generator=g))
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table, new_table = order[:B * per].view(B, per), order[B * per:B * (per + new)].view(B, new).contiguous()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return cache, mass, table, i32(lens), i32(keep), new_table


def reference(cache, mass, table, lens, keep, new_table, recent, first):
    """What stays, by a sort on the host: (new_lens, kept, the tensors after)."""
    B, H, page = len(lens), cache.k.shape[1], cache.k.shape[2]
    after = [t.clone() for t in (*cache, mass)]
    places = new_table.shape[1] * page
    kept = np.full((B, H, places), -1, dtype=np.int32)
    new_lens = []
    for b in range(B):
        L = int(lens[b])
        n = min(L, int(keep[b]))
        new_lens.append(n)
        last = min(recent, n)
        head = min(first, n - last)
        pos = torch.arange(L, device="cuda")
        src = table[b, pos // page].long()
        w = mass[src, :, pos % page].T.double().cpu().numpy()  # [H, L]
        w = np.where(np.isnan(w), -math.inf, w)
        for h in range(H):
            free = np.arange(head, L - last)
            best = free[np.argsort(-w[h, free], kind="stable")[:n - last - head]]
            stay = np.sort(np.concatenate([np.arange(head), best, np.arange(L - last, L)])).astype(np.int64)
            kept[b, h, :n] = stay
            at, i = torch.from_numpy(stay).cuda(), torch.arange(n, device="cuda")
            for t, old in zip(after, (*cache, mass)):
                t[new_table[b, i // page].long(), h, i % page] = old[table[b, at // page].long(), h, at % page]
    return torch.tensor(new_lens, dtype=torch.int32), torch.from_numpy(kept), after


def evict_and_check(fp8act, cache, mass, table, lens, keep, new_table, recent=0, first=0, **kw):  # noqa: F811
    want = reference(cache, mass, table, lens, keep, new_table, recent, first)
    new_lens, kept = fp8act.fp8_kv_evict(cache, mass, table, lens, keep, new_table, recent=recent, first=first, **kw)
    assert torch.equal(new_lens.cpu(), want[0]) and torch.equal(kept.cpu(), want[1])
    for got, ref in zip((*cache, mass), want[2]):
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))  # (bits: a scale may be anything)
    return new_lens, kept


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("H", [1, 3])
def test_evict(fp8act, D, page, H):  # noqa: F811
    lens = [1, 2, 63, 64, 65, 700, 4095, 4096, 4097, 0]
    keep = [1, 1, 62, 64, 1, 333, 4000, 1, 4097, 5]
    evict_and_check(fp8act, *problem(fp8act, lens, keep, H, D, page, seed=D + page), recent=7, first=3)


@pytest.mark.parametrize("L,keep", [(5000, 100), (20000, 19999), (131072, 8192), (131071, 1), (100003, 65537), (8200, 0)])
@pytest.mark.parametrize("H", [1, 4])
def test_evict_long_contexts(fp8act, L, keep, H):  # noqa: F811
    """Enough tokens for clusters of 2, 4 and 8 CTAs."""
    evict_and_check(fp8act, *problem(fp8act, [L], [keep], H, 64, 64, seed=L), recent=16, first=4)


def test_evict_more_tokens_than_shared_memory_holds(fp8act):  # noqa: F811
    evict_and_check(fp8act, *problem(fp8act, [400001], [300000], 1, 64, 256, seed=5), recent=100)
    lens = [41000, 50000] * 20 + [45000] * 60  # one CTA each
    evict_and_check(fp8act, *problem(fp8act, lens, [30] * 100, 1, 64, 256, seed=6))


@pytest.mark.parametrize("recent,first", [(0, 0), (50, 0), (0, 50), (30, 30), (1000, 5), (5, 1000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_evict_protected_tokens(fp8act, recent, first):  # noqa: F811
    lens, keep = [300, 40, 41, 100, 7], [40, 40, 40, 60, 3]
    evict_and_check(fp8act, *problem(fp8act, lens, keep, 2, 64, 16, seed=recent % 97 + first % 89), recent=recent, first=first)


def test_evict_ties_and_odd_weights(fp8act):  # noqa: F811
    lens, keep = [5000, 9000, 600, 300], [1234, 4000, 100, 299]
    cache, mass, table, lens, keep, new_table = problem(fp8act, lens, keep, 2, 64, 32, seed=8)
    for fill in (0.0, 1.0, math.nan, -math.inf, math.inf, 1e-45):
        mass.fill_(fill)
        evict_and_check(fp8act, cache, mass, table, lens, keep, new_table, recent=3)
    pool = torch.tensor([0.0, -0.0, 1.0, math.nan, math.inf, -math.inf, -1.0, 1e-45, 3e38, float(np.float32(1.0000001))], device="cuda")
    mass.copy_(pool[torch.randint(0, len(pool), mass.shape, device="cuda", generator=gen(9))])
    evict_and_check(fp8act, cache, mass, table, lens, keep, new_table, recent=3, first=2)
    mass.copy_((torch.randint(0, 3, mass.shape, device="cuda", generator=gen(10)) + (1 << 23)).int().view(torch.float32))
    evict_and_check(fp8act, cache, mass, table, lens, keep, new_table)  # neighbours in the last bit


@pytest.mark.parametrize("values", [1, 2, 5])
@pytest.mark.parametrize("L,keep", [(131071, 50001), (70000, 69999), (20011, 3)])
def test_evict_ties_in_long_contexts(fp8act, L, keep, values):  # noqa: F811
    """Of equal tokens the first stay, wherever among a sequence's CTAs and threads the last of them falls."""
    cache, mass, table, lens, keep, new_table = problem(fp8act, [L], [keep], 2, 64, 64, seed=values)
    mass.copy_(torch.randint(0, values, mass.shape, device="cuda", generator=gen(L)).float())
    evict_and_check(fp8act, cache, mass, table, lens, keep, new_table, recent=9, first=5)


def test_evict_leaves_the_old_pages(fp8act):  # noqa: F811
    """Two sequences that share a prefix are cut from the same old pages; again gives the same."""
    cache, mass, table, lens, keep, new_table = problem(fp8act, [200, 170], [64, 90], 2, 128, 16, seed=12)
    table = table.clone()
    table[1, :5] = table[0, :5]
    first = evict_and_check(fp8act, cache, mass, table, lens, keep, new_table, recent=8)
    again = evict_and_check(fp8act, cache, mass, table, lens, keep, new_table, recent=8)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_evict_index_errors(fp8act):  # noqa: F811
    cache, mass, table, lens, keep, new_table = problem(fp8act, [100, 100, 90], [40, 40, 40], 2, 64, 16, seed=14)
    want = reference(cache, mass, table, lens, keep, new_table, 0, 0)
    before = [t.clone() for t in (*cache, mass)]
    for name, bad in (("lens", 113), ("lens", -1), ("keep", 49), ("keep", -1)):
        a, k = lens.clone(), keep.clone()
        (a if name == "lens" else k)[1] = bad
        new_lens, kept = fp8act.fp8_kv_evict(cache, mass, table, a, k, new_table)
        assert fp8act.check_status() == INDEX and fp8act.check_status() == 0
        assert new_lens.tolist() == [40, {113: 40, -1: 0, 49: 48}[bad], 40]
        assert torch.equal(kept[0].cpu(), want[1][0]) and torch.equal(kept[2].cpu(), want[1][2])
    for t, old in zip((*cache, mass), before):
        t.copy_(old)
    for which in ("old", "new"):  # a page out of range: its tokens go last, or nowhere
        a, z = table.clone(), new_table.clone()
        (a if which == "old" else z)[1, 0] = len(cache.k)
        new_lens, kept = fp8act.fp8_kv_evict(cache, mass, a, lens, keep, z)
        assert fp8act.check_status() == INDEX and new_lens.tolist() == [40, 40, 40]
        assert torch.equal(kept[0].cpu(), want[1][0]) and torch.equal(kept[2].cpu(), want[1][2])
        assert which == "new" or (kept[1, :, :40] >= 16).all()


def test_evict_streams_graphs_and_nothing(fp8act):  # noqa: F811
    cache, mass, table, lens, keep, new_table = problem(fp8act, [9000, 300], [500, 20], 2, 64, 64, seed=16)
    cache.k[new_table.long()] = 0  # (places from n on are not written)
    want = evict_and_check(fp8act, cache, mass, table, lens, keep, new_table)
    fresh = cache.k[new_table.long()].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fp8act.fp8_kv_evict(cache, mass, table, lens, keep, new_table, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fp8act.fp8_kv_evict(cache, mass, table, lens, keep, new_table)
    for _ in range(2):
        cache.k[new_table.long()] = 0
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same = torch.equal(cache.k[new_table.long()], fresh)
        assert same and all(torch.equal(a, b) for a, b in zip(got, want))
    new_lens, kept = fp8act.fp8_kv_evict(cache, mass, table[:0], lens[:0], keep[:0], new_table[:0])
    assert new_lens.shape == (0,) and kept.shape == (0, 2, 512)
    new_lens, kept = fp8act.fp8_kv_evict(cache, mass, table, lens, torch.zeros_like(keep), new_table[:, :0].contiguous())
    assert new_lens.tolist() == [0, 0] and kept.shape == (2, 2, 0)


def test_evict_refusals(fp8act):  # noqa: F811
    cache, mass, table, lens, keep, new_table = problem(fp8act, [100], [40], 2, 64, 16, seed=18)
    a = (cache, mass, table, lens, keep, new_table)
    for i, bad in ((1, mass.double()), (2, table.long()), (3, lens.cpu()), (4, keep.float()), (5, new_table.long())):
        with pytest.raises(TypeError):
            fp8act.fp8_kv_evict(*a[:i], bad, *a[i + 1:])
    for i, bad in ((1, mass[:, :1]), (2, table[0]), (3, lens.repeat(2)), (5, new_table.repeat(2, 1)), (1, mass.transpose(1, 2))):
        with pytest.raises(ValueError):
            fp8act.fp8_kv_evict(*a[:i], bad, *a[i + 1:])
    for kw in (dict(recent=-1), dict(first=-1), dict(new_lens=lens), dict(new_lens=keep)):
        with pytest.raises(fp8act.Fp8ActError):
            fp8act.fp8_kv_evict(*a, **kw)
    with pytest.raises(ValueError):
        fp8act.fp8_kv_evict(*a, recent=1 << 40)
