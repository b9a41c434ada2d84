"""GPU tests of fp8_rope_append at the ends of its range: heads whose squares or weighted values pass fp32's, and positions
whose angles pass fp64's. Tolerances as in test_gpu_rope_append.py, with the angle's own stated where it counts."""
from __future__ import annotations

import math
from fractions import Fraction

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


def turns_of(positions, inv_freq):
    """The angles as fractions of a turn in [-1/2, 1/2), exact but for 2^-200 of a turn a radian."""
    def arctan(n, one):  # of 1 / n
        power = total = one // n
        k, sign = 1, 1
        while power:
            power //= n * n
            k, sign = k + 2, -sign
            total += sign * (power // k)
        return total

    one = 1 << 320
    pi = 4 * (4 * arctan(5, one) - arctan(239, one))  # (Machin)
    turn = Fraction(one, 2 * pi)
    out = [[(Fraction(f) * p * turn + Fraction(1, 2)) % 1 - Fraction(1, 2) for f in inv_freq] for p in positions]
    return torch.tensor([[float(x) for x in row] for row in out], dtype=torch.float64, device="cuda")


@pytest.mark.parametrize("theta", [1e4, 1e7])
@pytest.mark.parametrize("most", [1 << 20, 1 << 45, 1 << 50, 1 << 55, 1 << 62])
def test_rope_angles_of_far_positions(fp8act, most, theta):  # noqa: F811
    """Against exact angles of the given frequencies: off by |position| 2^-64 turns (a frequency is a whole number of those a
    position) and 2^-62 of the angle, beside what any angle is off by."""
    T, Hq, D = 48, 4, 64
    q, k, v = randn(T, Hq, D, seed=1), randn(T, 1, D, seed=2), randn(T, 1, D, seed=3)
    inv = theta ** (-2.0 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
    inv[5] = -inv[5]
    pos = torch.randint(0, most, (T,), device="cuda", generator=gen(4)) * torch.where(torch.arange(T, device="cuda") % 3 > 0, 1, -1)
    out = fp8act.fp8_rope_append(q, k, v, pos, inv, torch.full((T,), -1, device="cuda"), fp8act.kv_cache(1, 1, 16, D)).double()
    angle = 2 * math.pi * turns_of(pos.tolist(), inv.tolist()).unsqueeze(1)
    a, b = q.double()[..., :D // 2], q.double()[..., D // 2:]
    want = torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)
    p = pos.double().abs().view(T, 1, 1)
    off = 2 * math.pi * 2.0 ** -64 * p + 2.0 ** -62 * p * inv.abs()
    tol = ((a.abs() + b.abs()) * (2.0 ** -18 + off)).repeat(1, 1, 2)
    assert ((out - want).abs() <= 2.0 ** -8 * want.abs() + tol).all()
