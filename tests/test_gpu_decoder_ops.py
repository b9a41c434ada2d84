"""GPU tests of the operators between the linear layers, each against its
definition in 64 bits on the same inputs.

Tolerances, from the arithmetic:
* norm, silu: y carries at most 64 fp32 roundings (a sum of K squares in
  partial sums of at most 32 terms and two 32-wide trees, a reciprocal root,
  three products; an exponential, a quotient, a product), so scales agree to
  2^-18 and a code is the E4M3 of some value within 2^-17 of y / s;
* append: bit-exact with the IEEE quotient;
* attention: |error| <= 2^-8 |o| + 2^-10 sum p |v|. bf16 rounds o by 2^-9 |o|;
  the weights' f16 rounding adds 2^-12 sum p |v|, and a score's fp32 error
  (D products of size <= 16: below 2^-13) twice that much of sum p |v|;
* verification: an accepted count or a token may differ only where the
  decision's own margin is below 1e-5 (64 fp32 roundings and the
  exponential's argument of at most 100 rounded to 2^-24).
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

G = 128
INDEX = 8  # FP8ACT_ERR_INDEX


@pytest.fixture(scope="module")
def fp8act():
    from block_scaled_fp8_act_gb300 import fp8act as mod
    mod.load(build=True)
    return mod


@pytest.fixture(autouse=True)
def clean_status(fp8act):
    yield
    assert fp8act.check_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, seed, scale=1.0):
    return (scale * torch.randn(shape, device="cuda", generator=gen(seed))).bfloat16()


def e4m3(x):
    """fp64 -> the nearest E4M3 value (fp64), ties to even, saturating."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def check_codes(q, sa, y):
    """q, sa [M, K], [M, K/128] against fp64 y."""
    M, K = y.shape
    yg = y.view(M, K // G, G)
    amax = yg.abs().amax(-1)
    ref = torch.where(amax > 0, amax / 448.0, 1.0)
    assert ((sa.double() - ref).abs() <= 2.0 ** -18 * ref).all()
    r = yg / ref.unsqueeze(-1)
    got = q.view(torch.float8_e4m3fn).double().view_as(r)
    lo, hi = e4m3(r * (1 - 2.0 ** -17)), e4m3(r * (1 + 2.0 ** -17))
    assert ((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))).all()


# ------------------------------------------------------------------- norm
def norm_ref(x, w, residual, eps, offset):
    h = x.double() if residual is None else x.double() + residual.double()
    return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * (w.double() + offset)


@pytest.mark.parametrize("M,K", [(1, 128), (1, 5120), (3, 384), (2, 8192), (5, 8320), (2, 32768), (305, 5120),
                                 (1000, 1152), (700, 128)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_rmsnorm(fp8act, M, K, with_residual):
    x, w = randn(M, K, seed=M + K), randn(K, seed=7)
    r = randn(M, K, seed=3, scale=5.0) if with_residual else None
    got = fp8act.fp8_rmsnorm_quant(x, w, residual=r, eps=1e-5, weight_offset=1.0)
    check_codes(got[0], got[1], norm_ref(x, w, r, 1e-5, 1.0))
    if with_residual:
        assert torch.equal(got[2], (x.float() + r.float()).bfloat16())


def test_rmsnorm_in_place_empty_and_zero_rows(fp8act):
    x, w = randn(9, 640, seed=1), randn(640, seed=2)
    r = randn(9, 640, seed=3)
    x[4] = 0
    r[4] = 0
    x[5], r[6] = 1e-30, 3e4
    want = fp8act.fp8_rmsnorm_quant(x, w, residual=r)
    check_codes(want[0], want[1], norm_ref(x, w, r, 1e-6, 0.0))
    assert (want[1][4] == 1).all() and (want[0][4] & 0x7F == 0).all()
    r2 = r.clone()
    got = fp8act.fp8_rmsnorm_quant(x, w, residual=r2, residual_out=r2)
    assert got[2] is r2 and all(torch.equal(a, b) for a, b in zip(got, want))
    q, sa = fp8act.fp8_rmsnorm_quant(x[:0], w)
    assert q.shape == (0, 640) and sa.shape == (0, 5)


def test_rmsnorm_feeds_the_gemm(fp8act):
    """Its codes and scales are the block GEMM's activation operands."""
    x, w = randn(4, 512, seed=5), randn(512, seed=6)
    W = randn(256, 512, seed=8, scale=0.05)
    q, sa = fp8act.fp8_rmsnorm_quant(x, w)
    wq, sw = fp8act.fp8_weight_quant(W)
    out = fp8act.fp8_block_gemm_f32(q, sa, wq, sw)
    a = q.view(torch.float8_e4m3fn).double() * sa.double().repeat_interleave(G, 1)
    b = wq.view(torch.float8_e4m3fn).double() * sw.double().repeat_interleave(G, 0).repeat_interleave(G, 1)
    want = a @ b.T
    assert (out.double() - want).norm() <= 1e-4 * want.norm()


# ------------------------------------------------------------------- silu
@pytest.mark.parametrize("M,n", [(1, 128), (1, 8704), (8, 1152), (77, 384), (1000, 640)])
def test_silu_mul(fp8act, M, n):
    x = randn(M, 2 * n, seed=M + n, scale=3.0)
    q, sa = fp8act.fp8_silu_mul_quant(x)
    g, u = x.double().chunk(2, -1)
    check_codes(q, sa, g * torch.sigmoid(g) * u)


def test_silu_extremes(fp8act):
    x = torch.zeros((4, 256), device="cuda", dtype=torch.bfloat16)
    x[:, 128:] = 1.0
    x[0, :8] = torch.tensor([-3e38, -200.0, -88.0, -1.0, 0.0, 1.0, 88.0, 200.0], device="cuda").bfloat16()
    x[1, :128] = -200.0     # all but vanishing
    x[2, 128:] = 0.0        # an all-zero group
    x[3, :128] = 3e4
    q, sa = fp8act.fp8_silu_mul_quant(x)
    v = q.view(torch.float8_e4m3fn).double() * sa.double()
    want = x[:, :128].double() * torch.sigmoid(x[:, :128].double()) * x[:, 128:].double()
    assert torch.isfinite(v).all()
    assert ((v - want).abs() <= want.abs().amax(-1, keepdim=True) * 2.0 ** -4 + 1e-30).all()
    assert (sa[2] == 1).all()


# ------------------------------------------------------------------ cache
def quant_ref(x):
    """The IEEE rule on the CPU: codes (uint8) and scales of bf16 vectors along the last axis."""
    x = x.float().cpu()
    amax = x.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones(()), amax / torch.full((), 448.0))
    return (x / s.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (37, 3, 32), (500, 4, 64), (9, 8, 256)])
def test_append_bit_exact(fp8act, T, H, page, D):
    rows = randn(T, 3 * H * D + 8, seed=T * D, scale=2.0)  # keys and values are columns of wider rows
    rows *= torch.exp2(torch.randint(-20, 20, (T, 1), device="cuda", generator=gen(4))).bfloat16()
    k, v = rows[:, 8:8 + H * D].unflatten(1, (H, D)), rows[:, 8 + 2 * H * D:].unflatten(1, (H, D))
    k[0, 0] = 0
    cache = fp8act.kv_cache(T // page + 3, H, page, D)
    for t in cache:
        t.fill_(77)
    slots = torch.randperm((T // page + 3) * page, device="cuda", generator=gen(5))[:T]
    slots[T // 2] = -1 if T > 1 else slots[T // 2]
    fp8act.fp8_kv_append(k, v, slots, cache)
    want = [t.cpu().clone().fill_(77) for t in cache]
    keep = (slots >= 0).cpu()
    at = slots.cpu()[keep]
    for x, codes, scales in ((k, want[0], want[2]), (v, want[1], want[3])):
        q, s = quant_ref(x)
        codes[at // page, :, at % page] = q[keep]
        scales[at // page, :, at % page] = s[keep]
    for got, ref in zip(cache, want):
        assert torch.equal(got.cpu(), ref)


def test_append_every_bf16_pair_of_a_vector(fp8act):
    """Scales and codes on the whole exponent range, subnormals included."""
    bits = torch.arange(0x7F80, dtype=torch.int32)
    x = torch.zeros((0x7F80, 1, 64), dtype=torch.bfloat16)
    x[:, 0, 0] = bits.to(torch.int16).view(torch.bfloat16)
    fill = torch.randint(0, 0x7F80, (0x7F80, 63), generator=torch.Generator().manual_seed(1)) % (bits + 1).unsqueeze(1)
    x[:, 0, 1:] = (fill | (torch.arange(63) % 2 * 0x8000)).to(torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x.cuda()
    cache = fp8act.kv_cache(0x7F80 // 16, 1, 16, 64)
    slots = torch.arange(0x7F80, device="cuda")
    fp8act.fp8_kv_append(x, x, slots, cache)
    q, s = quant_ref(x[:, 0])
    assert torch.equal(cache.k.view(-1, 64).cpu() & 0x7F, q & 0x7F)
    assert torch.equal(cache.k_scale.view(-1).cpu(), s) and torch.equal(cache.k, cache.v)


def test_append_non_finite_and_out_of_range(fp8act):
    x = randn(4, 2, 128, seed=9)
    x[1, 0, 5], x[2, 1, 0] = math.nan, math.inf
    cache = fp8act.kv_cache(2, 2, 16, 128)
    fp8act.fp8_kv_append(x, x, torch.tensor([0, 1, 2, 32], device="cuda"), cache)
    assert fp8act.check_status() == INDEX and fp8act.check_status() == 0  # slot 32 is past the two pages
    bad = torch.isnan(cache.k_scale)
    assert bad.sum() == 2 and bad[0, 0, 1] and bad[0, 1, 2]
    assert (cache.k[bad] == 0).all() and not torch.isnan(cache.k.view(torch.float8_e4m3fn).float()).any()
    assert (cache.k[1] == 0).all()
    fp8act.fp8_kv_append(x[:0], x[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), cache)


def test_append_and_attend_past_four_gigabytes(fp8act):
    H, page, D = 8, 256, 256
    pages = (1 << 32) // (H * page * D) + 2
    cache = fp8act.kv_cache(pages, H, page, D)
    assert cache.k.numel() > 1 << 32
    k, v, q = randn(3, H, D, seed=1), randn(3, H, D, seed=2), randn(3, 2 * H, D, seed=3)
    at = (pages - 1) * page + torch.arange(3, device="cuda")
    fp8act.fp8_kv_append(k, v, at, cache)
    codes, s = quant_ref(k)
    assert torch.equal(cache.k[pages - 1, :, :3].transpose(0, 1).cpu(), codes)
    table = torch.full((1, 1), pages - 1, dtype=torch.int32, device="cuda")
    attend_and_check(fp8act, q, cache, table, [3], [3])


# -------------------------------------------------------------- attention
def make_cache(fp8act, lens, H, D, page, seed, v_scale=None):
    """A cache of random keys and values; slots that hold no token are NaN."""
    per = max(1, max(-(-max(n, 1) // page) for n in lens))
    B = len(lens)
    pages = B * per + 2
    cache = fp8act.kv_cache(pages, H, page, D)
    cache.k.fill_(0x7F)
    cache.v.fill_(0xFF)
    cache.k_scale.fill_(math.nan)
    cache.v_scale.fill_(math.nan)
    table = torch.randperm(pages, device="cuda", generator=gen(seed))[:B * per].view(B, per).to(torch.int32)
    total = sum(lens)
    k, v = randn(total, H, D, seed=seed + 1, scale=1.5), randn(total, H, D, seed=seed + 2)
    if v_scale is not None:
        v *= v_scale(total).view(-1, 1, 1).bfloat16()
    slots = torch.cat([table[b].long().repeat_interleave(page)[:n] * page + torch.arange(n, device="cuda") % page
                       for b, n in enumerate(lens)]) if total else torch.zeros(0, dtype=torch.int64, device="cuda")
    fp8act.fp8_kv_append(k, v, slots, cache)
    return cache, table


def attention_ref(q, cache, table, lens, ns, scale):
    """fp64 output, sum p |v|, and lse."""
    T, Hq, D = q.shape
    H, page = cache.k.shape[1], cache.k.shape[2]
    out, mag = torch.zeros((2, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (L, n) in enumerate(zip(lens, ns)):
        at = table[b, :-(-L // page)].long()
        k, v = ((c[at].view(torch.float8_e4m3fn).double() * s[at].double().unsqueeze(-1)).transpose(1, 2).flatten(0, 1)[:L]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        k, v = k.repeat_interleave(Hq // H, 1), v.repeat_interleave(Hq // H, 1)
        for i in range(n):
            see = L - n + i + 1
            if see <= 0:
                continue
            x = torch.einsum("hd,lhd->hl", q[t0 + i].double(), k[:see]) * scale
            p = torch.softmax(x, -1)
            out[t0 + i] = torch.einsum("hl,lhd->hd", p, v[:see])
            mag[t0 + i] = torch.einsum("hl,lhd->hd", p, v[:see].abs())
            lse[t0 + i] = torch.logsumexp(x, -1)
        t0 += n
    return out, mag, lse


def attend(fp8act, q, cache, table, lens, ns, **kw):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw.setdefault("max_q_len", max(ns))
    return fp8act.fp8_kv_attention(q, cache, table, kv, cu, **kw)


def check_attention(out, ref, mag):
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag).all(), float((err / (mag + 1e-30)).max())


def attend_and_check(fp8act, q, cache, table, lens, ns, **kw):
    lse = torch.empty(q.shape[:2], device="cuda")
    out = attend(fp8act, q, cache, table, lens, ns, lse=lse, **kw)
    ref, mag, lref = attention_ref(q, cache, table, lens, ns, kw.get("softmax_scale") or q.shape[2] ** -0.5)
    check_attention(out, ref, mag)
    empty = lref == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (out[empty] == 0).all()
    assert ((lse.double() - lref)[~empty].abs() <= 2.0 ** -12 + 2.0 ** -20 * lref[~empty].abs()).all()
    return out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group,n", [(1, 1), (6, 1), (3, 2), (6, 3), (12, 3), (6, 8), (8, 8), (5, 40)])
def test_attention_head_layouts(fp8act, D, group, n):
    H = 2
    lens = [n, 63 + n, 64, 65, 130, 1000]
    ns = [min(n, L) for L in lens]
    cache, table = make_cache(fp8act, lens, H, D, 16, seed=D + group)
    q = randn(sum(ns), H * group, D, seed=3)
    attend_and_check(fp8act, q, cache, table, lens, ns)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("L", [1, 15, 16, 17, 255, 256, 257, 5000])
def test_attention_lengths_and_pages(fp8act, page, L):
    cache, table = make_cache(fp8act, [L], 1, 128, page, seed=L + page)
    attend_and_check(fp8act, randn(1, 4, 128, seed=L), cache, table, [L], [1])


def test_attention_rows_that_see_nothing(fp8act):
    lens, ns = [0, 2, 5, 0, 70], [3, 5, 0, 1, 2]  # no cache, more new tokens than cached, no new tokens
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=11)
    out = attend_and_check(fp8act, randn(sum(ns), 6, 128, seed=12), cache, table, lens, ns)
    assert (out[:3] == 0).all() and (out[3:6] == 0).all() and (out[8] == 0).all()


def test_attention_large_ragged_batch(fp8act):
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 900, 70)]
    ns = [min(int(x), L) for x, L in zip(rng.integers(0, 9, 70), lens)]
    cache, table = make_cache(fp8act, lens, 2, 64, 32, seed=13)
    q = randn(sum(ns), 6, 64, seed=14)
    first = attend_and_check(fp8act, q, cache, table, lens, ns)
    for hint in (1, 4, 100):  # the hint changes the row tile, not the result
        attend_and_check(fp8act, q, cache, table, lens, ns, max_q_len=hint)
    again = attend(fp8act, q, cache, table, lens, ns)
    assert torch.equal(first, again)


@pytest.mark.parametrize("D,n", [(128, 1), (128, 8), (64, 300), (128, 300), (256, 150)])
def test_attention_long_context_and_chunks(fp8act, D, n):
    L = 9000 if n < 100 else 700
    cache, table = make_cache(fp8act, [L], 2, D, 64, seed=n)
    attend_and_check(fp8act, randn(n, 8, D, seed=n), cache, table, [L], [n])


def test_attention_whole_prompt(fp8act):
    cache, table = make_cache(fp8act, [333, 64], 2, 128, 16, seed=1)  # every token new: fully causal
    attend_and_check(fp8act, randn(397, 4, 128, seed=2), cache, table, [333, 64], [333, 64])


def test_attention_peaked_scores_and_uneven_scales(fp8act):
    """Scores of +-100 and value scales over 2^24: the maximum moves often, and so does the weights' scale."""
    def v_scale(total):
        return torch.exp2(torch.randint(-12, 13, (total,), device="cuda", generator=gen(5)).float())
    lens, ns = [777, 300], [4, 1]
    cache, table = make_cache(fp8act, lens, 2, 128, 32, seed=6, v_scale=v_scale)
    attend_and_check(fp8act, randn(5, 8, 128, seed=7), cache, table, lens, ns, softmax_scale=1.0)
    attend_and_check(fp8act, randn(5, 8, 128, seed=7, scale=1e-30), cache, table, lens, ns)
    attend_and_check(fp8act, torch.zeros_like(randn(5, 8, 128, seed=7)), cache, table, lens, ns)


# Row tiles from 49 rows on, head size 128: the tcgen05 kernel, with one row tile (up to 128 rows), two halves of one
# (up to 256), and several. Its values are widened with their scales, to within 2^-31 of the largest scale's power of
# two, R: an absolute error of at most 2^-30 of the sequence's largest |v| beside the others.
WIDE = [(9, 6), (64, 2), (22, 6), (32, 8), (43, 6), (100, 7)]


@pytest.mark.parametrize("n,group", WIDE)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attention_wide_row_tiles(fp8act, n, group, page):
    lens = [n, 127, 128, 129, 1, 700, 0, 2500]
    ns = [min(n, L) if i % 2 == 0 else n for i, L in enumerate(lens)]  # some with more new tokens than cached
    cache, table = make_cache(fp8act, lens, 2, 128, page, seed=n + page)
    q = randn(sum(ns), 2 * group, 128, seed=3)
    first = attend_and_check(fp8act, q, cache, table, lens, ns)
    assert torch.equal(attend(fp8act, q, cache, table, lens, ns), first)


@pytest.mark.parametrize("n,group", [(20, 6), (60, 6)])
def test_attention_wide_rows_peaked_scores_and_uneven_scales(fp8act, n, group):
    def v_scale(total):
        return torch.exp2(torch.randint(-12, 13, (total,), device="cuda", generator=gen(5)).float())
    lens, ns = [777, 300], [n, n // 2]
    cache, table = make_cache(fp8act, lens, 2, 128, 32, seed=6, v_scale=v_scale)
    for scale, softmax_scale in ((1.0, 1.0), (1e-30, None), (0.0, None)):
        q = randn(sum(ns), 2 * group, 128, seed=7, scale=scale)
        out = attend(fp8act, q, cache, table, lens, ns, softmax_scale=softmax_scale)
        ref, mag, _ = attention_ref(q, cache, table, lens, ns, softmax_scale or 128 ** -0.5)
        vmax = 448.0 * float(cache.v_scale.nan_to_num(0.0).max())
        assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag + 2.0 ** -30 * vmax).all()


def test_attention_wide_rows_long_context_and_batch(fp8act):
    lens, ns = [9000], [16]
    cache, table = make_cache(fp8act, lens, 2, 128, 64, seed=61)
    attend_and_check(fp8act, randn(16, 12, 128, seed=62), cache, table, lens, ns)
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(1, 1500, 40)]
    ns = [min(int(x), L) for x, L in zip(rng.integers(0, 40, 40), lens)]
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=63)
    q = randn(sum(ns), 8, 128, seed=64)
    for hint in (20, 100):  # one row tile of 80 rows, or 256
        attend_and_check(fp8act, q, cache, table, lens, ns, max_q_len=hint)


def test_attention_wide_rows_nan_query(fp8act):
    lens, ns = [500], [20]
    cache, table = make_cache(fp8act, lens, 2, 128, 16, seed=65)
    q = randn(20, 12, 128, seed=66)
    clean = attend(fp8act, q, cache, table, lens, ns)
    q[7, 3, 5], q[9, 11, 0] = math.nan, math.inf
    out = attend(fp8act, q, cache, table, lens, ns)
    bad = torch.isnan(out).all(-1)
    assert bad.sum() == 2 and bad[7, 3] and bad[9, 11]
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("n", [16, 60])
def test_attention_wait_that_runs_out(fp8act, n):
    """The tcgen05 kernel leaves cleanly when a copy never comes, and the next call is right."""
    lens, ns = [3000, 100], [n, n]
    cache, table = make_cache(fp8act, lens, 2, 128, 64, seed=71)
    q = randn(2 * n, 12, 128, seed=72)
    want = attend_and_check(fp8act, q, cache, table, lens, ns)
    try:
        fp8act.set_wait_limit(1_000_000, True)
        attend(fp8act, q, cache, table, lens, ns)
        assert fp8act.check_status() == 5  # FP8ACT_ERR_TIMEOUT
        fp8act.set_wait_limit(0, False)
        attend(fp8act, q, cache, table, lens, ns)
        assert fp8act.check_status() in (0, 5)
    finally:
        fp8act.set_wait_limit(-1, False)
    assert torch.equal(attend(fp8act, q, cache, table, lens, ns), want)


@pytest.mark.parametrize("n", [3, 40, 100])
def test_attention_nan_reaches_only_rows_that_see_it(fp8act, n):
    L, H = 100, 2
    cache, table = make_cache(fp8act, [L], H, 128, 16, seed=21)
    q = randn(n, 6, 128, seed=22)
    clean = attend(fp8act, q, cache, table, [L], [n])
    x = randn(1, H, 128, seed=23)
    x[0, 0, 3] = math.nan  # KV head 0 of the last cached token
    slot = table[0, (L - 1) // 16].long() * 16 + (L - 1) % 16
    keep = tuple(t.clone() for t in cache)
    for bad in ("k", "v"):
        for t, s in zip(cache, keep):
            t.copy_(s)
        spare = tuple(t.clone() for t in cache)
        fp8act.fp8_kv_append(x, x, slot.view(1), cache)
        for i in ((1, 3) if bad == "k" else (0, 2)):  # poison only one of the two
            cache[i].copy_(spare[i])
        out = attend(fp8act, q, cache, table, [L], [n])
        assert torch.equal(out[:-1], clean[:-1])
        assert torch.isnan(out[-1, :3]).all() and torch.isfinite(out[-1, 3:]).all()


def test_attention_strided_queries_stream_and_workspace(fp8act):
    lens, ns, H, D = [400, 90], [2, 1], 2, 128
    cache, table = make_cache(fp8act, lens, H, D, 64, seed=31)
    rows = randn(3, 1536, seed=32)
    q = rows[:, 256:256 + 6 * D].unflatten(1, (6, D))
    want = attend_and_check(fp8act, q, cache, table, lens, ns)
    assert torch.equal(attend(fp8act, q.contiguous(), cache, table, lens, ns), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    need = fp8act.kv_attention_workspace(2, 6, cache)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [attend(fp8act, q, cache, table, lens, ns, workspace=ws) for _ in range(5)]
    side.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with pytest.raises(fp8act.Fp8ActError):
        attend(fp8act, q, cache, table, lens, ns, workspace=ws[:-16])


def test_attention_indices_out_of_range(fp8act):
    lens, ns = [100, 100], [1, 1]
    cache, table = make_cache(fp8act, lens, 1, 128, 16, seed=41)
    q = randn(2, 2, 128, seed=42)
    want = attend(fp8act, q, cache, table, lens, ns)
    bad = table.clone()
    bad[1, 2] = 1 << 30
    out = attend(fp8act, q, cache, bad, lens, ns)
    assert fp8act.check_status() == INDEX
    assert torch.equal(out[0], want[0])
    attend(fp8act, q, cache, table, [100, 1 << 30], ns)       # longer than the page table: cut to it
    assert fp8act.check_status() == INDEX
    out = torch.full_like(q, 7.0)
    attend(fp8act, q, cache, table, lens, [1, 100], out=out, max_q_len=1)  # cu_q past q: that sequence is left out
    assert fp8act.check_status() == INDEX
    assert torch.equal(out[0], want[0]) and (out[1] == 7).all()


def test_append_and_attention_in_a_graph(fp8act):
    H, D, page, L = 2, 128, 16, 50
    cache, table = make_cache(fp8act, [L], H, D, page, seed=51)
    k, v, q = randn(2, H, D, seed=52), randn(2, H, D, seed=53), randn(2, 6, D, seed=54)
    slots = table[0, 3].long() * page + torch.tensor([0, 1], device="cuda")
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    kv = torch.tensor([50], dtype=torch.int32, device="cuda")
    ws = torch.zeros(fp8act.kv_attention_workspace(2, 6, cache), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step():
        fp8act.fp8_kv_append(k, v, slots, cache)
        fp8act.fp8_kv_attention(q, cache, table, kv, cu, max_q_len=2, out=out, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        k.copy_(randn(2, H, D, seed=seed))
        q.copy_(randn(2, 6, D, seed=seed + 10))
        graph.replay()
        ref, mag, _ = attention_ref(q, cache, table, [50], [2], D ** -0.5)
        check_attention(out, ref, mag)


# ----------------------------------------------------------- verification
def verify_ref(target, draft, x, u, e, temp, n):
    """One sequence in 64 bits: (accepted, tokens, probabilities, smallest margin of a decision)."""
    k, V = x.numel(), target.shape[1]
    greedy = not temp > 0

    def soft(row):
        row = torch.where(torch.isnan(row), -math.inf, row.double())
        if greedy:
            p = torch.zeros_like(row)
            if row.max() > -math.inf:
                p[int((row == row.max()).nonzero()[0])] = 1.0
            return p
        if not row.max() > -math.inf:
            return torch.zeros_like(row)
        return torch.softmax(row / temp, -1)
    margin, probs, a, stopped = 1.0, [0.0] * k, 0, False
    for j in range(n):
        p = soft(target[j])[x[j]]
        q = 1.0 if draft is None or greedy else soft(draft[j])[x[j]]
        probs[j] = float(min(p / q, 1.0)) if q > 0 else float(p > 0)
        if not stopped:
            if not greedy:
                margin = min(margin, abs(float(u[j]) - probs[j]))
            stopped = not float(u[j]) < probs[j]
            a += not stopped
    p = soft(target[a])
    w = p
    if a < n and not greedy:
        q = torch.zeros_like(p)
        if draft is None:
            q[x[a]] = 1.0
        else:
            q = soft(draft[a])
        w = (p - q).clamp(min=0)
        if not (w > 0).any():
            w = p
    key = torch.where(w > 0, w / e.double(), -1.0)
    token = int((key == key.max()).nonzero()[0]) if key.max() > 0 else -1
    return a, [int(v) for v in x[:a]] + [token] + [-1] * (k - a), probs, margin, key


def check_verify(fp8act, target, draft, x, u, e, temp, n=None):
    got = fp8act.verify_drafts(target, x, u, e, temp, draft_logits=draft, n_draft=n)
    took, tokens, prob = (t.cpu() for t in got)
    B, k = x.shape
    for b in range(B):
        a, want, probs, margin, key = verify_ref(target[b].cpu().double(), None if draft is None else draft[b].cpu().double(),
                                                 x[b].cpu(), u[b].cpu(), e[b].cpu(), float(temp[b]),
                                                 k if n is None else int(n[b]))
        assert np.allclose(prob[b].numpy(), probs, rtol=1e-5, atol=1e-12), b
        if margin < 1e-5:
            continue
        assert int(took[b]) == a, b
        t = tokens[b].tolist()
        assert t[:a] == want[:a] and t[a + 1:] == want[a + 1:], b
        if t[a] != want[a]:  # two draws that fp32 cannot tell apart
            assert t[a] >= 0 and float(key[t[a]]) >= (1 - 1e-5) * float(key.max()), b
    return got


def drafts(B, k, V, seed, dtype=torch.bfloat16, err=0.5):
    g = gen(seed)
    t = 3.0 * torch.randn((B, k + 1, V), device="cuda", generator=g)
    d = t[:, :k] + err * torch.randn((B, k, V), device="cuda", generator=g)
    t, d = t.to(dtype), d.to(dtype)
    race = torch.empty((B, k, V), device="cuda").exponential_(generator=g)
    x = (d.float().softmax(-1) / race).argmax(-1).to(torch.int32)
    u = torch.rand((B, k), device="cuda", generator=g)
    e = torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_(min=1e-20)
    return t, d, x, u, e


@pytest.mark.parametrize("V", [1, 2, 7, 17, 1001, 4096, 33333, 151936])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_verify_vocabularies(fp8act, V, dtype):
    t, d, x, u, e = drafts(5, 3, V, seed=V, dtype=dtype)
    temp = torch.tensor([1.0, 0.7, 0.0, 1.3, 0.3], device="cuda")
    check_verify(fp8act, t, d, x, u, e, temp)
    check_verify(fp8act, t, None, t[:, :3].float().argmax(-1).to(torch.int32), u, e, temp)


@pytest.mark.parametrize("k", [0, 1, 7, 31, 32])
@pytest.mark.parametrize("B", [1, 40])
def test_verify_draft_lengths(fp8act, B, k):
    t, d, x, u, e = drafts(B, k, 2222, seed=B + k, err=0.1)
    u *= 0.5  # long runs of acceptances
    n = torch.randint(0, k + 1, (B,), device="cuda", generator=gen(1)).to(torch.int32)
    check_verify(fp8act, t, d, x, u, e, torch.full((B,), 0.9, device="cuda"), n)
    check_verify(fp8act, t, d, x, u, e, torch.zeros(B, device="cuda"))


def test_verify_masks(fp8act):
    t, d, x, u, e = drafts(8, 2, 5000, seed=77, dtype=torch.float32)
    t[0] = -math.inf                                    # nothing left in any row
    t[1, 0] = -math.inf                                 # nothing left in the first
    t[2] = torch.where(t[2] > 2, t[2], -math.inf)       # a cut to the likely tokens
    t[3] = torch.where(t[3] > 2, t[3], math.nan)        # the same with NaN
    t[4] = torch.where(t[4] > 2, t[4], torch.finfo(torch.float32).min)
    t[5, :, :] = -math.inf
    t[5, :, 4321] = 1.0                                 # one token left
    d[6] = t[6, :2]                                     # drafts from the target itself: always accepted
    t[7, 0, x[7, 0]] = -math.inf                        # the drafted token is masked
    temp = torch.ones(8, device="cuda")
    took, tokens, prob = check_verify(fp8act, t, d, x, u, e, temp)
    assert tokens[0].tolist() == [-1, -1, -1] and tokens[1].tolist() == [-1, -1, -1]
    assert int(tokens[5, int(took[5])]) == 4321 and took[6] == 2 and took[7] == 0
    took, tokens, _ = check_verify(fp8act, t, d, x, u, e, 0 * temp)
    assert tokens[0].tolist() == [-1, -1, -1]


def test_verify_ties_and_equal_models(fp8act):
    B, V = 4, 3000
    t = torch.zeros((B, 2, V), device="cuda", dtype=torch.bfloat16)
    x = torch.full((B, 1), 9, dtype=torch.int32, device="cuda")
    e = torch.ones((B, V), device="cuda")
    u = torch.full((B, 1), 0.5, device="cuda")
    temp = torch.tensor([1.0, 1.0, 0.0, 0.0], device="cuda")
    x[2] = 0
    took, tokens, _ = fp8act.verify_drafts(t, x, u, e, temp, draft_logits=t[:, :1].contiguous())
    # equal logits: p = q accepts, the draw goes to the lowest of equal keys; greedy picks token 0
    assert took.tolist() == [1, 1, 1, 0] and tokens[:, 0].tolist() == [9, 9, 0, 0] and tokens[:3, 1].tolist() == [0, 0, 0]


def test_verify_token_out_of_range(fp8act):
    t, d, x, u, e = drafts(2, 2, 100, seed=5)
    x[0, 0], x[1, 0] = 100, -3
    took, tokens, prob = fp8act.verify_drafts(t, x, u, e, torch.ones(2, device="cuda"), draft_logits=d)
    assert fp8act.check_status() == INDEX
    assert took.tolist() == [0, 0] and prob[:, 0].tolist() == [0, 0] and (tokens[:, 0] >= 0).all()
    fp8act.verify_drafts(t, x.clamp(0, 99), u, e, torch.ones(2, device="cuda"), draft_logits=d,
                         n_draft=torch.tensor([3, -1], dtype=torch.int32, device="cuda"))
    assert fp8act.check_status() == INDEX


@pytest.mark.parametrize("greedy_draft", [False, True])
def test_verify_keeps_the_targets_distribution(fp8act, greedy_draft):
    """Whatever drafted it, the first token is distributed as the target's softmax (chi-square over 6 tokens, 5 sigma)."""
    B, V = 60000, 6
    g = gen(99)
    t = torch.tensor([0.3, -1.0, 1.1, 0.0, -2.0, 0.6], device="cuda").expand(B, 2, V).contiguous()
    d = torch.tensor([1.0, 0.5, -0.5, 0.0, 0.2, 0.1], device="cuda").expand(B, 1, V).contiguous()
    race = torch.empty((B, 1, V), device="cuda").exponential_(generator=g)
    x = (d.softmax(-1) / race).argmax(-1).to(torch.int32)
    if greedy_draft:
        d, x = None, torch.full_like(x, 2)
    u = torch.rand((B, 1), device="cuda", generator=g)
    e = torch.empty((B, V), device="cuda").exponential_(generator=g)
    _, tokens, _ = fp8act.verify_drafts(t, x, u, e, torch.ones(B, device="cuda"), draft_logits=d)
    want = t[0, 0].double().softmax(-1) * B
    seen = torch.bincount(tokens[:, 0].long(), minlength=V).double()
    chi2 = float(((seen - want) ** 2 / want).sum())
    assert chi2 < (V - 1) + 5 * math.sqrt(2 * (V - 1)) + 25


def test_verify_right_behind_its_producers(fp8act):
    """Logits come from two products just before, step after step without a pause; nothing old may be read."""
    B, k, V, K = 2, 3, 4096, 256
    w, sw = fp8act.fp8_weight_quant(randn(V, K, seed=1))
    acts = [(fp8act.fp8_act_quant(randn(B * (k + 1), K, seed=10 + i)), fp8act.fp8_act_quant(randn(B * k, K, seed=20 + i)))
            for i in range(3)]
    _, _, x, u, e = drafts(B, k, V, seed=3)
    temp = torch.tensor([1.0, 0.6], device="cuda")
    t = torch.empty((B * (k + 1), V), dtype=torch.bfloat16, device="cuda")
    d = torch.empty((B * k, V), dtype=torch.bfloat16, device="cuda")

    def step(i, pause):
        fp8act.fp8_block_gemm(*acts[i][1], w, sw, out=d)
        fp8act.fp8_block_gemm(*acts[i][0], w, sw, out=t)
        if pause:
            torch.cuda.synchronize()
        return fp8act.verify_drafts(t.view(B, k + 1, V), x, u, e, temp, draft_logits=d.view(B, k, V))

    want = [step(i, True) for i in range(3)]
    torch.cuda.synchronize()
    got = [step(i % 3, False) for i in range(30)]
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3]))


def test_kept_workspace_grows_on_a_stream_that_is_passed(fp8act):
    """A call that needs more memory than the one before lets the old go while the stream still works on it."""
    side = torch.cuda.Stream()
    small, large = drafts(1, 1, 5000, seed=1), drafts(40, 7, 5000, seed=2)
    temp = [torch.ones(1, device="cuda"), torch.ones(40, device="cuda")]

    def call(s, t, **kw):
        return fp8act.verify_drafts(s[0], s[2], s[3], s[4], t, draft_logits=s[1], **kw)

    want = call(small, temp[0]), call(large, temp[1])
    torch.cuda.synchronize()
    got = call(small, temp[0], stream=side), call(large, temp[1], stream=side)
    # the current stream asks for memory of the old one's size and writes it
    junk = [torch.full((512,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    side.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w)) and len(junk) == 8


@pytest.mark.parametrize("n", [1, 2, 4, 9, 30])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_one_long_context_and_short_ones(fp8act, D, n):
    """Items of tens of parts, joined by several warps a row, next to items of one part and to empty sequences."""
    lens, ns = [9000, 0, 33, 700], [n, 0, 1, 2]
    cache, table = make_cache(fp8act, lens, 2, D, 64, seed=61)
    q = randn(sum(ns), 2 * 6, D, seed=62)
    attend_and_check(fp8act, q, cache, table, lens, ns)
    # fewer tokens announced than a sequence has: other row tiles, the same attention
    attend_and_check(fp8act, q, cache, table, lens, ns, max_q_len=max(1, n // 3))
    one, table = make_cache(fp8act, [20000], 1, D, 64, seed=63)
    q = randn(n, 6, D, seed=64)
    attend_and_check(fp8act, q, one, table, [20000], [n])
    attend_and_check(fp8act, q, one, table, [20000], [n], max_q_len=1)
