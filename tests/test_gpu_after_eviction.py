"""GPU test of what distances mean after an eviction: window, documents and bias count places of the cache, not the positions
that its tokens once had. Tolerances as in test_gpu_scores.py."""
from __future__ import annotations

import pytest
import torch
from test_gpu_decoder_ops import attend, clean_status, fp8act, gen, make_cache, randn  # noqa: F401  (fixtures too)
from test_gpu_scores import check, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
def test_distances_are_places(fp8act, D):  # noqa: F811
    H, page, lens, keep = 2, 16, [400, 300], [90, 120]
    cache, table = make_cache(fp8act, lens, H, D, page, seed=D)
    old = len(cache.k)
    cache = fp8act.KvCache(*(torch.cat([t, torch.zeros_like(t[:16])]) for t in cache))  # fresh pages
    fresh = torch.arange(old, old + 16, dtype=torch.int32, device="cuda").view(2, 8)
    mass = torch.rand(cache.k_scale.shape, device="cuda", generator=gen(1))
    new_lens, kept = fp8act.fp8_kv_evict(cache, mass, table, i32(lens), i32(keep), fresh, recent=4)
    assert new_lens.tolist() == keep
    # the last places are the last positions; before them lie older tokens, closer together than they were, in each head others
    n, ns = keep, [1, 2]
    assert (kept[0, :, n[0] - 4:n[0]].cpu() == torch.arange(396, 400)).all()
    assert (kept[0, :, n[0] - 20] < 380).all() and not torch.equal(kept[0, 0], kept[0, 1])
    q = randn(3, 6 * H, D, seed=2)
    for how in (dict(window=30), dict(slopes=torch.linspace(0.01, 0.5, 6 * H, device="cuda")), dict(first=i32([60, 100, 100]))):
        check(fp8act, q, cache, fresh, n, ns, **how)  # (the definition with i and j places)
