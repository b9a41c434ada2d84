"""GPU tests of the head norms, rotary positions and cache append in one pass,
against the definition in 64 bits on the same inputs.

Tolerances, from the arithmetic. A normed value carries the sum of squares (14
fp32 roundings, halved by the root), the reciprocal root (2 ulp) and three more
roundings: below 2^-20 of it. Cosine and sine are off by the angle's rounding to
fp32 (2^-25 of at most pi), the function's (2 ulp), and twice 2^-52 of the angle
itself, once here and once in the reference; the turn adds two products and a
sum. A turned value is thus within 2^-18 (|a| + |b|) of the pair's exact one,
plus 2^-50 |angle| (|a| + |b|). Queries are rounded to bf16, 2^-8 of the value.
The largest pair has |a| + |b| <= 2 amax, so that scales agree to 2^-17 and a
code is the E4M3 of some value within 2^-16 * 448 of y / s.
"""
from __future__ import annotations

import math

import pytest
import torch
from test_gpu_decoder_ops import INDEX, clean_status, e4m3, fp8act, gen, randn  # noqa: F401  (fixtures too)

pytestmark = pytest.mark.gpu


def rope_ref(x, weight, positions, inv_freq, axes, interleaved, eps=1e-6, offset=0.0, scale=1.0):
    """fp64 result, its tolerance before rounding; x [T, H, D]."""
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * (weight.double() + offset)
    half = len(inv_freq)
    pos = positions if positions.dim() == 2 else positions.unsqueeze(0)
    axis = torch.zeros(half, dtype=torch.long, device="cuda") if axes is None else axes.long()
    angle = (pos[axis].T.double() * inv_freq).unsqueeze(1)  # [T, 1, half]
    at = torch.arange(half, device="cuda")
    i, j = (2 * at, 2 * at + 1) if interleaved else (at, at + half)
    a, b = x[..., i], x[..., j]
    y, tol = x.clone(), x.abs() * 2.0 ** -18
    y[..., i] = scale * (a * torch.cos(angle) - b * torch.sin(angle))
    y[..., j] = scale * (a * torch.sin(angle) + b * torch.cos(angle))
    both = scale * (a.abs() + b.abs())
    tol[..., i] = tol[..., j] = both * (2.0 ** -18 + 2.0 ** -50 * angle.abs())
    return y, tol


def check_cached(codes, s, y, tol):
    """codes, s [T, H, D], [T, H] against fp64 y."""
    amax = y.abs().amax(-1)
    ref = torch.where(amax > 0, amax / 448.0, 1.0)
    most = tol.amax(-1) / 448.0 + 2.0 ** -22 * ref
    assert ((s.double() - ref).abs() <= most).all()
    r, near = y / ref.unsqueeze(-1), (448.0 * most / ref).unsqueeze(-1) + tol / ref.unsqueeze(-1)
    got = codes.view(torch.float8_e4m3fn).double()
    assert ((got >= e4m3(r - near)) & (got <= e4m3(r + near))).all()


def problem(T, Hq, H, D, rot, axes, norm, seed, most=100000):
    rows = randn(T, (Hq + 2 * H) * D + 8, seed=seed, scale=2.0)  # columns of wider rows
    q, k, v = (t.unflatten(1, (-1, D)) for t in rows[:, 8:].split([Hq * D, H * D, H * D], 1))
    qw, kw = (randn(D, seed=seed + i) if norm else None for i in (1, 2))
    inv = 1e6 ** (-2.0 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / max(rot, 1))
    pos = torch.randint(0, most, (axes, T), device="cuda", generator=gen(seed + 3))
    axis = torch.randint(0, axes, (rot // 2,), device="cuda", generator=gen(seed + 4)).to(torch.int32)
    return q, k, v, qw, kw, inv, pos, axis


def filled(fp8act, pages, H, page, D):  # noqa: F811
    cache = fp8act.kv_cache(pages, H, page, D)
    for t in cache:
        t.fill_(77)
    return cache


@pytest.mark.parametrize("T,Hq,H,D,rot,axes,norm,interleaved,page", [
    (1, 24, 4, 128, 128, 1, True, False, 64), (1, 1, 1, 64, 64, 1, True, False, 16), (3, 5, 1, 256, 256, 2, True, True, 32),
    (37, 6, 3, 64, 48, 3, False, False, 16), (37, 6, 3, 64, 16, 1, True, True, 128), (102, 24, 4, 128, 64, 3, True, False, 16),
    (9, 7, 7, 256, 240, 4, False, False, 256), (5, 40, 8, 128, 112, 2, True, True, 64), (700, 12, 2, 128, 128, 3, True, False, 64),
    (650, 3, 1, 64, 64, 1, True, True, 32), (4, 130, 2, 256, 32, 1, True, False, 16), (2, 3, 2, 128, 0, 1, True, False, 16),
    # many tokens: two a round, or as many as a warp has room for
    (4097, 24, 4, 128, 128, 3, True, False, 64), (6001, 1, 1, 64, 64, 1, True, False, 16), (6003, 2, 1, 64, 32, 2, True, True, 32),
    (5001, 3, 1, 64, 48, 1, False, False, 16), (4003, 1, 1, 128, 128, 2, True, True, 64), (4999, 2, 2, 128, 64, 1, True, False, 16),
    (3001, 1, 1, 256, 256, 3, True, False, 16), (2999, 2, 2, 256, 128, 1, True, True, 256), (1501, 40, 8, 64, 64, 4, True, False, 16)])
def test_rope_append(fp8act, T, Hq, H, D, rot, axes, norm, interleaved, page):  # noqa: F811
    q, k, v, qw, kw, inv, pos, axis = problem(T, Hq, H, D, rot, axes, norm, seed=T + D)
    pages = T // page + 2
    cache = filled(fp8act, pages, H, page, D)
    plain = filled(fp8act, pages, H, page, D)
    slots = torch.randperm(pages * page, device="cuda", generator=gen(5))[:T]
    if T > 2:
        slots[1] = -1
    how = dict(q_weight=qw, k_weight=kw, eps=1e-5, weight_offset=1.0, interleaved=interleaved, rope_scale=1.25)
    if axes == 1:
        pos, axis = pos[0], None
    out = fp8act.fp8_rope_append(q, k, v, pos, inv, slots, cache, axes=axis, **how)
    args = (pos, inv, axis, interleaved, 1e-5, 1.0, 1.25)
    want, tol = rope_ref(q, qw, *args)
    assert out.shape == q.shape and ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + tol).all()
    fp8act.fp8_kv_append(k, v, slots, plain)
    assert torch.equal(cache.v, plain.v) and torch.equal(cache.v_scale, plain.v_scale)
    there = slots >= 0
    at = slots[there]
    want, tol = rope_ref(k, kw, *args)
    check_cached(cache.k[at // page, :, at % page], cache.k_scale[at // page, :, at % page], want[there], tol[there])
    untouched = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    untouched[at] = False
    untouched = untouched.view(pages, page)
    assert (cache.k.transpose(1, 2)[untouched] == 77).all() and (cache.k_scale.transpose(1, 2)[untouched] == 77).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rope_of_nothing_is_the_append(fp8act, D):  # noqa: F811
    """No norm and no rotated columns, or position 0: queries and keys pass as they are."""
    T, Hq, H = 41, 6, 2
    q, k, v, _, _, inv, pos, _ = problem(T, Hq, H, D, D, 1, False, seed=3)
    slots = torch.randperm(64, device="cuda", generator=gen(1))[:T]
    want = fp8act.kv_cache(4, H, 16, D)
    fp8act.fp8_kv_append(k, v, slots, want)
    for p, f in ((pos[0], inv[:0]), (torch.zeros_like(pos[0]), inv)):
        cache = fp8act.kv_cache(4, H, 16, D)
        out = fp8act.fp8_rope_append(q, k, v, p, f, slots, cache)
        assert torch.equal(out, q) and all(torch.equal(a, b) for a, b in zip(cache, want))


@pytest.mark.parametrize("most", [1 << 20, 1 << 30, 1 << 40])
def test_rope_far_and_negative_positions(fp8act, most):  # noqa: F811
    q, k, v, qw, kw, inv, pos, _ = problem(64, 2, 1, 64, 64, 1, True, seed=9, most=most)
    pos[0, ::2] *= -1
    cache = fp8act.kv_cache(4, 1, 16, 64)
    out = fp8act.fp8_rope_append(q, k, v, pos[0], inv, torch.arange(64, device="cuda"), cache, q_weight=qw, k_weight=kw)
    want, tol = rope_ref(q, qw, pos, inv, None, False)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + tol).all()
    # a frequency of a whole turn and a quarter is a quarter
    f = torch.full((32,), 2 * math.pi * 1.25, dtype=torch.float64, device="cuda")
    g = torch.full((32,), 2 * math.pi * 0.25, dtype=torch.float64, device="cuda")
    small = torch.arange(64, device="cuda") - 32
    a, b = (fp8act.fp8_rope_append(q, k, v, small, x, torch.arange(64, device="cuda"), cache).double() for x in (f, g))
    want, tol = rope_ref(q, None, small, g, None, False)
    for y in (a, b):
        assert ((y - want).abs() <= 2.0 ** -8 * want.abs() + tol + 2.0 ** -42).all()


def test_rope_non_finite_and_zero_heads(fp8act):  # noqa: F811
    q, k, v, qw, kw, inv, pos, _ = problem(5, 4, 2, 128, 64, 1, True, seed=21)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    k[1, 0, 5], k[2, 1, 100], v[3, 0, 7] = math.nan, math.inf, -math.inf
    q[4, 2, 9] = math.nan
    k[0, 0] = 0
    q[0, 1] = 0
    cache = fp8act.kv_cache(1, 2, 16, 128)
    out = fp8act.fp8_rope_append(q, k, v, pos[0], inv, torch.arange(5, device="cuda"), cache, q_weight=qw, k_weight=kw)
    bad = torch.isnan(cache.k_scale)
    assert bad.sum() == 2 and bad[0, 0, 1] and bad[0, 1, 2] and (cache.k[bad] == 0).all()
    bad = torch.isnan(cache.v_scale)
    assert bad.sum() == 1 and bad[0, 0, 3] and (cache.v[bad] == 0).all()
    assert (cache.k[0, 0, 0] & 0x7F == 0).all() and cache.k_scale[0, 0, 0] == 1 and (out[0, 1] == 0).all()
    nan = torch.isnan(out)
    assert nan[4, 2].all() and nan.sum() == 128


def test_rope_index_errors(fp8act):  # noqa: F811
    q, k, v, _, _, inv, pos, axis = problem(4, 2, 2, 64, 32, 2, False, seed=31)
    axis.zero_()
    cache = filled(fp8act, 2, 2, 16, 64)
    want = fp8act.fp8_rope_append(q, k, v, pos, inv, torch.tensor([0, 1, 2, -5], device="cuda"), cache, axes=axis)
    got = filled(fp8act, 2, 2, 16, 64)
    out = fp8act.fp8_rope_append(q, k, v, pos, inv, torch.tensor([0, 1, 2, 32], device="cuda"), got, axes=axis)
    assert fp8act.check_status() == INDEX and fp8act.check_status() == 0
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(cache, got))
    for bad in (2, -1):  # no such axis: the first one's position
        axis[3] = bad
        out = fp8act.fp8_rope_append(q, k, v, pos, inv, torch.tensor([0, 1, 2, -5], device="cuda"), got, axes=axis)
        assert fp8act.check_status() == INDEX and torch.equal(out, want)


def test_rope_streams_graphs_and_no_tokens(fp8act):  # noqa: F811
    q, k, v, qw, kw, inv, pos, _ = problem(33, 6, 2, 128, 128, 1, True, seed=41)
    cache = fp8act.kv_cache(4, 2, 16, 128)
    slots = torch.arange(33, device="cuda")
    call = lambda c=cache, **kw2: fp8act.fp8_rope_append(q, k, v, pos[0], inv, slots, c, q_weight=qw, k_weight=kw, **kw2)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fp8act.kv_cache(4, 2, 16, 128)
    got = call(other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(cache, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(other)
    for t in other:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a[:2], b[:2]) for a, b in zip(cache, other))
    empty = fp8act.fp8_rope_append(q[:0], k[:0], v[:0], pos[0, :0], inv, slots[:0], cache)
    assert empty.shape == (0, 6, 128)


def test_rope_binding_refusals(fp8act):  # noqa: F811
    q, k, v, qw, kw, inv, pos, axis = problem(4, 2, 2, 64, 32, 2, True, seed=51)
    cache = fp8act.kv_cache(2, 2, 16, 64)
    slots = torch.arange(4, device="cuda")

    def call(**kw2):
        a = dict(q=q, k=k, v=v, positions=pos, inv_freq=inv, slots=slots, cache=cache, axes=axis)
        a.update(kw2)
        return fp8act.fp8_rope_append(**a)
    call()
    for bad in (dict(inv_freq=inv.float()), dict(positions=pos.int()), dict(slots=slots.int()), dict(q=q.float()),
                dict(axes=axis.long()), dict(q_weight=qw.float()), dict(slots=slots.cpu())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(positions=pos[:, :3]), dict(k=k[:3]), dict(k=k[:, :1]), dict(axes=axis[:3]), dict(slots=slots[:3]),
                dict(q=q[..., :32]), dict(q_weight=qw[:32]), dict(positions=pos.view(2, 2, 2)),
                dict(q_out=torch.empty((4, 2, 128), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(inv_freq=inv[:9].clone(), axes=None), dict(inv_freq=torch.zeros(40, dtype=torch.float64, device="cuda"), axes=None),
                dict(positions=pos.repeat(3, 1)), dict(positions=pos[:0].contiguous())):
        with pytest.raises(fp8act.Fp8ActError):
            call(**bad)


@pytest.mark.parametrize("T,Hq,H,D,interleaved", [(1301, 24, 4, 128, False), (2999, 5, 3, 64, True), (3000, 1, 1, 64, False), (1500, 3, 3, 256, True)])
def test_rope_many_tokens_are_as_few(fp8act, T, Hq, H, D, interleaved):  # noqa: F811
    """However the tokens are shared out, their bits are those of calls with a few: among slots left out and heads of zeros,
    infinities and NaN."""
    q, k, v, qw, kw, inv, pos, axis = problem(T, Hq, H, D, D, 2, True, seed=T)
    g = gen(T)
    for x in (q, k, v):
        for odd in (0.0, math.inf, math.nan, 1e-40, 3e38):
            x[torch.randint(0, T, (20,), device="cuda", generator=g), torch.randint(0, x.shape[1], (20,), device="cuda", generator=g)] = odd
    pages = T // 16 + 2
    slots = torch.randperm(pages * 16, device="cuda", generator=g)[:T]
    slots[torch.randint(0, T, (T // 10,), device="cuda", generator=g)] = -1
    got, few = filled(fp8act, pages, H, 16, D), filled(fp8act, pages, H, 16, D)
    how = dict(axes=axis, q_weight=qw, k_weight=kw, interleaved=interleaved)
    out = fp8act.fp8_rope_append(q, k, v, pos, inv, slots, got, **how)
    for i in range(0, T, 97):
        at = slice(i, i + 97)
        part = fp8act.fp8_rope_append(q[at], k[at], v[at], pos[:, at].contiguous(), inv, slots[at], few, **how)
        assert torch.equal(out[at].view(torch.int16), part.view(torch.int16))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, few))
