"""GPU tests of fp8_rope_append at the ends of its range: heads whose squares or weighted values pass fp32's, and positions
whose angles pass fp64's. Tolerances as in test_gpu_rope_append.py, with the angle's own stated where it counts."""
from __future__ import annotations

import pytest
import torch
from test_gpu_decoder_ops import clean_status, fp8act, gen, randn  # noqa: F401  (fixtures too)
from test_gpu_rope_append import check_cached, problem, rope_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4, 3000])  # (one token a warp, and two at a time)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rope_of_heads_whose_squares_overflow(fp8act, D, interleaved, T):  # noqa: F811
    """In fp32 the mean of their squares is infinite and its reciprocal root zero: the head becomes zeros, whatever the weight."""
    Hq, H = 6, 2
    q, k, v, qw, kw, inv, pos, _ = problem(T, Hq, H, D, D, 1, True, seed=D)
    q, k = q.contiguous(), k.contiguous()
    for x in (q, k):
        x[1] = (3e38 * torch.sign(x[1].float())).bfloat16()  # (times a weight above 1.13: past the range)
        x[2, :, 5], x[2, :, D // 2 + 3] = 3e38, -1e30
    qw, kw = ((2 + w.float().abs()).bfloat16() for w in (qw, kw))
    cache = fp8act.kv_cache(T // 16 + 1, H, 16, D)
    slots = torch.arange(T, device="cuda")
    out = fp8act.fp8_rope_append(q, k, v, pos[0], inv, slots, cache, q_weight=qw, k_weight=kw, interleaved=interleaved)
    codes, s = cache.k[slots // 16, :, slots % 16], cache.k_scale[slots // 16, :, slots % 16]
    assert (out[1:3] == 0).all() and (codes[1:3] & 0x7F == 0).all() and (s[1:3] == 1).all()
    there = torch.ones(T, dtype=torch.bool, device="cuda")
    there[1:3] = False
    want, tol = rope_ref(q, qw, pos[0], inv, None, interleaved)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + tol)[there].all()
    want, tol = rope_ref(k, kw, pos[0], inv, None, interleaved)
    check_cached(codes[there], s[there], want[there], tol[there])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rope_of_heads_whose_weighted_values_overflow(fp8act, D):  # noqa: F811
    """Values of 1e15 with weights of 1e25: the product is past fp32's range, the normed value is not."""
    T, Hq, H = 40, 6, 2
    q, k, v, qw, kw, inv, pos, _ = problem(T, Hq, H, D, D, 1, True, seed=D + 1)
    q, k = ((x.float() * 1e15).bfloat16() for x in (q, k))
    qw, kw = ((w.float() * 1e25).bfloat16() for w in (qw, kw))
    cache = fp8act.kv_cache(3, H, 16, D)
    slots = torch.arange(T, device="cuda")
    out = fp8act.fp8_rope_append(q, k, v, pos[0], inv, slots, cache, q_weight=qw, k_weight=kw)
    want, tol = rope_ref(q, qw, pos[0], inv, None, False)
    assert torch.isfinite(out).all() and ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + tol).all()
    want, tol = rope_ref(k, kw, pos[0], inv, None, False)
    check_cached(cache.k[slots // 16, :, slots % 16], cache.k_scale[slots // 16, :, slots % 16], want, tol)
