"""GPU test of rows that see nothing but tokens far away: their biases are thousands, and so are their scores.

A biased score is off by the product's 2^-13 (test_gpu_decoder_ops.py) and 2^-21 of its bias: the slope's two roundings and
its constant's, the multiply-add's, the unit's of a cap and the exponent's, each 2^-24 of it. Weights are off by twice that
relative to themselves, since the sum has it too (and lse, to which weights of tokens are taken, once more its own 2^-24).
"""
from __future__ import annotations

import pytest
import torch
from test_gpu_decoder_ops import attend, clean_status, fp8act, make_cache, randn  # noqa: F401  (fixtures too)
from test_gpu_scores import i32, scores_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("n", [1, 8, 30])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_that_see_far_tokens_alone(fp8act, D, n, cap):  # noqa: F811
    H, group, L = 2, 6, 6000
    cache, table = make_cache(fp8act, [L], H, D, 64, seed=D + n)
    q = randn(n, H * group, D, seed=n)
    slopes = torch.linspace(0.01, 1.0, H * group, device="cuda")
    how = dict(prefix_lens=i32([40]), first=i32([L + 5] * n), slopes=slopes, soft_cap=cap)
    lse = torch.empty((n, H * group), device="cuda")
    out = attend(fp8act, q, cache, table, [L], [n], lse=lse, **how).double()
    mass = fp8act.kv_mass(cache)
    fp8act.fp8_kv_attention_mass(q, cache, table, i32([L]), i32([0, n]), lse, mass, max_q_len=n, accumulate=False, **how)
    (_, x, v), = scores_ref(q, cache, table, [L], [n], D ** -0.5, **how)
    bias = slopes.double() * L
    p = torch.softmax(x, -1)
    ref, mag = (torch.einsum("nhl,lhd->nhd", p, t) for t in (v, v.abs()))
    assert ((out - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2.0 ** -20 * bias).view(1, -1, 1) * mag).all()
    want = torch.logsumexp(x, -1)
    assert ((lse.double() - want).abs() <= 2.0 ** -12 + 2.0 ** -21 * bias + 2.0 ** -23 * want.abs()).all()
    w = torch.exp(x - lse.double().unsqueeze(-1))[..., :40].unflatten(1, (H, group))
    tol = ((2.0 ** -12 + 2.0 ** -20 * bias).view(1, H, group, 1) * w).sum((0, 2))
    got = mass[table[0, 0].long(), :, :40].double()
    assert ((got - w.sum((0, 2))).abs() <= tol + 1e-30).all()
