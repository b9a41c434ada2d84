"""GPU tests of the operators between the linear layers where a caller's memory,
streams or values are unusual: views at odd offsets, streams that are passed,
producers right in front, ends of the number range."""
from __future__ import annotations

import pytest
import torch
from test_gpu_decoder_ops import (check_verify, clean_status, drafts, e4m3, fp8act, gen,  # noqa: F401  (fixtures too)
                                  randn)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------- verification: noise
@pytest.mark.parametrize("V", [8, 4096, 5000, 151936])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_verify_noise_at_any_offset(fp8act, V, dtype):  # noqa: F811
    """Noise cut out of a larger buffer need not start on a 16-byte boundary; the draw is the aligned one's."""
    B, k = 4, 2
    t, d, x, u, e = drafts(B, k, V, seed=V, dtype=dtype)
    temp = torch.tensor([1.0, 0.7, 0.0, 1.3], device="cuda")
    want = check_verify(fp8act, t, d, x, u, e, temp)
    assert e.data_ptr() % 16 == 0
    for offset in (1, 2, 3):
        buffer = torch.full((B * V + 4,), float("nan"), device="cuda")
        view = buffer[offset:offset + B * V].view(B, V)
        view.copy_(e)
        assert view.data_ptr() % 16 == 4 * offset
        for draft in (d, None):
            got = check_verify(fp8act, t, draft, x, u, view, temp)
            if draft is not None:
                assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_verify_right_behind_the_writers_of_its_small_inputs(fp8act):  # noqa: F811
    """Tokens, numbers, temperatures, counts and noise are written just before, step after step without a pause."""
    B, k, V = 3, 4, 5000
    steps = []
    for i in range(3):
        t, d, x, u, e = drafts(B, k, V, seed=100 + i, err=0.2)
        temp = torch.tensor([1.0, 0.0, 0.5], device="cuda").roll(i)
        n = torch.tensor([k, 2, 3], dtype=torch.int32, device="cuda").roll(i)
        steps.append((t, d, x, u * 0.5, e, temp, n))
    now = [torch.empty_like(a) for a in steps[0]]

    def step(i, pause):
        for dst, src in zip(now, steps[i]):
            dst.copy_(src)
        if pause:
            torch.cuda.synchronize()
        return fp8act.verify_drafts(now[0], now[2], now[3], now[4], now[5], draft_logits=now[1], n_draft=now[6])

    want = [step(i, True) for i in range(3)]
    for w, (t, d, x, u, e, temp, n) in zip(want, steps):
        got = check_verify(fp8act, t, d, x, u, e, temp, n)
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    got = [step(i % 3, False) for i in range(60)]
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3]))


# ------------------------------------------------------------------- norm
@pytest.mark.parametrize("M,K", [(1, 5120), (300, 1152), (2, 16384)])
def test_rmsnorm_right_behind_the_writer_of_its_weight(fp8act, M, K):  # noqa: F811
    """The weight may be a cast just made, with one of the library's own kernels between or none."""
    x = randn(M, K, seed=1)
    weights = [randn(K, seed=10 + i).float() for i in range(3)]
    want = [fp8act.fp8_rmsnorm_quant(x, w.bfloat16()) for w in weights]
    torch.cuda.synchronize()
    w = torch.empty(K, dtype=torch.bfloat16, device="cuda")
    got = []
    for i in range(60):
        w.copy_(weights[i % 3])
        if i & 1:
            fp8act.fp8_act_quant(x)  # lets the kernel behind it start at once
        got.append(fp8act.fp8_rmsnorm_quant(x, w))
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3]))


# ---------------------------------------------------------------- streams
def segment_stream(t):
    """The stream whose memory pool holds `t`."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not in any segment")


def allocated(stream):
    return sum(s["allocated_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == stream)


def busy(x, n):
    """Some milliseconds of work on the current stream."""
    for _ in range(n):
        x = torch.tanh(x)
    return x


def verify_problem(B, k, V, seed):
    t, d, x, u, e = drafts(B, k, V, seed=seed)
    return (t, x, u, e, torch.ones(B, device="cuda")), d


def test_memory_made_for_a_passed_stream_is_from_its_pool(fp8act):  # noqa: F811
    side = torch.cuda.Stream()
    x, w = randn(3, 640, seed=1), randn(640, seed=2)
    cache = fp8act.kv_cache(2, 1, 16, 64)
    q = randn(1, 2, 64, seed=3)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    args, draft = verify_problem(2, 2, 1000, 4)
    torch.cuda.synchronize()
    calls = [lambda **kw: fp8act.fp8_rmsnorm_quant(x, w, x, **kw), lambda **kw: fp8act.fp8_silu_mul_quant(x[:, :512].contiguous(), **kw),
             lambda **kw: (fp8act.fp8_kv_attention(q, cache, table, lens, cu, **kw),),
             lambda **kw: fp8act.verify_drafts(*args, draft_logits=draft, **kw)]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        for stream in (side, side.cuda_stream):
            got = call(stream=stream)
            assert all(segment_stream(t) == side.cuda_stream for t in got)
            torch.cuda.current_stream().wait_stream(side)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(segment_stream(t) == torch.cuda.current_stream().cuda_stream for t in want)


def test_kept_workspace_is_the_streams_own(fp8act):  # noqa: F811
    """However the calls come, passed or current, a stream's workspace and its growth stay in that stream's pool."""
    side = torch.cuda.Stream()
    (small, ds), (large, dl) = verify_problem(1, 1, 3000, 1), verify_problem(60, 7, 3000, 2)
    outs = [dict(accepted=torch.empty(B, dtype=torch.int32, device="cuda"),
                 tokens=torch.empty((B, k + 1), dtype=torch.int32, device="cuda"),
                 accept_prob=torch.empty((B, k), device="cuda")) for B, k in ((1, 1), (60, 7))]
    main = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    before = allocated(main)
    fp8act.verify_drafts(*small, draft_logits=ds, **outs[0], stream=side)
    first = allocated(side.cuda_stream)
    with torch.cuda.stream(side):
        fp8act.verify_drafts(*large, draft_logits=dl, **outs[1])
    second = allocated(side.cuda_stream)
    side.synchronize()
    assert allocated(main) <= before  # (less if something old is collected meanwhile)
    assert 0 < fp8act.verify_drafts_workspace(1, 1) <= first and fp8act.verify_drafts_workspace(60, 7) <= second


def test_growth_under_the_stream_itself_while_it_works(fp8act):  # noqa: F811
    """First call by a passed stream, second under it: the workspace that is let go must not reach another stream."""
    side = torch.cuda.Stream()
    (small, ds), (large, dl) = verify_problem(1, 1, 5000, 1), verify_problem(40, 7, 5000, 2)
    want = fp8act.verify_drafts(*small, draft_logits=ds), fp8act.verify_drafts(*large, draft_logits=dl)
    x = randn(4096, 4096, seed=3)
    size = fp8act.verify_drafts_workspace(1, 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        held = busy(x, 200)
    first = fp8act.verify_drafts(*small, draft_logits=ds, stream=side)
    with torch.cuda.stream(side):
        second = fp8act.verify_drafts(*large, draft_logits=dl)
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip((first, second), want) for a, b in zip(g, w))
    assert len(junk) == 64 and held.shape == x.shape


def test_memory_that_the_current_stream_still_uses(fp8act):  # noqa: F811
    """Blocks freed on the current stream with writes to them still queued there are not what a passed stream gets."""
    side = torch.cuda.Stream()
    args, draft = verify_problem(9, 3, 5000, 5)
    want = fp8act.verify_drafts(*args, draft_logits=draft)
    x = randn(4096, 4096, seed=3)
    sizes = [fp8act.verify_drafts_workspace(9, 3)] + [t.numel() * t.element_size() for t in want]
    torch.cuda.synchronize()
    held = busy(x, 200)
    for _ in range(16):
        for n in sizes:
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # freed at once, written late
    got = [fp8act.verify_drafts(*args, draft_logits=draft, stream=side) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want)) and held.shape == x.shape


def test_outputs_dropped_while_their_stream_works(fp8act):  # noqa: F811
    side = torch.cuda.Stream()
    args, draft = verify_problem(9, 3, 5000, 6)
    want = fp8act.verify_drafts(*args, draft_logits=draft)
    x = randn(4096, 4096, seed=3)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        held = busy(x, 200)
    took, tokens, _ = fp8act.verify_drafts(*args, draft_logits=draft, stream=side)
    junk = [torch.full((9, 3), 7.0, device="cuda") for _ in range(64)]
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(took, want[0]) and torch.equal(tokens, want[1])
    assert all((j == 7).all() for j in junk) and held.shape == x.shape


def test_capture_on_a_passed_stream(fp8act):  # noqa: F811
    """In a capture that the current stream has no part in, outputs and workspace must be brought; then it replays."""
    args, draft = verify_problem(3, 2, 2000, 7)
    want = fp8act.verify_drafts(*args, draft_logits=draft)
    outs = dict(zip(("accepted", "tokens", "accept_prob"), (torch.zeros_like(t) for t in want)))
    ws = torch.empty(fp8act.verify_drafts_workspace(3, 2), dtype=torch.uint8, device="cuda")
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            with pytest.raises(ValueError):
                fp8act.verify_drafts(*args, draft_logits=draft, stream=side)
            with pytest.raises(ValueError):
                fp8act.verify_drafts(*args, draft_logits=draft, **outs, stream=side)
            fp8act.verify_drafts(*args, draft_logits=draft, **outs, workspace=ws, stream=side)
    for _ in range(2):
        for t in outs.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs.values(), want))


def test_fork_inside_a_capture(fp8act):  # noqa: F811
    """A stream that joined torch's capture may be passed; the graph owns what the calls make."""
    args, draft = verify_problem(3, 2, 2000, 8)
    x, w = randn(5, 640, seed=1), randn(640, seed=2)
    want = *fp8act.verify_drafts(*args, draft_logits=draft), *fp8act.fp8_rmsnorm_quant(x, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = *fp8act.verify_drafts(*args, draft_logits=draft, stream=side), *fp8act.fp8_rmsnorm_quant(x, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        junk = [torch.full((1 << 12,), 255, dtype=torch.uint8, device="cuda") for _ in range(16)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 16


# ------------------------------------------------------------------- silu
def test_silu_of_gates_with_a_large_exponential(fp8act):  # noqa: F811
    """Down to where exp(-gate) overflows the gate's share is still a normal number, and a large `up` shows it.

    An exponent of up to 128 is rounded by 2^-18 and the constant's error adds 2^-19, times ln 2: a relative error
    below 2^-17 with the other roundings."""
    gates = [-88.5, -88.0, -87.5, -87.0, -80.0, -60.0, -20.0]
    x = torch.empty((len(gates), 256), device="cuda")
    x[:, :128] = torch.tensor(gates, device="cuda").view(-1, 1)
    x[:, 128:] = 2e38 * (2 * torch.rand((len(gates), 128), device="cuda", generator=gen(3)) - 1)
    x[-1, 128:] *= 1e-10
    x = x.bfloat16()
    q, sa = fp8act.fp8_silu_mul_quant(x)
    g, u = x.double().chunk(2, -1)
    y = g * torch.sigmoid(g) * u
    want = y.abs().amax(-1, keepdim=True) / 448.0
    assert (want > 0.02).all() and ((sa.double() - want).abs() <= 2.0 ** -17 * want).all()
    r, got = y / want, q.view(torch.float8_e4m3fn).double()
    lo, hi = e4m3(r * (1 - 2.0 ** -16)), e4m3(r * (1 + 2.0 ** -16))
    assert ((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))).all()
    x[:, :128] = -89.0  # exp(89) is infinite in fp32
    q, sa = fp8act.fp8_silu_mul_quant(x)
    assert (q & 0x7F == 0).all() and (sa == 1).all()


# ---------------------------------------------- verification: temperatures
@pytest.mark.parametrize("V", [4096, 5001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_verify_ends_of_the_temperature_range(fp8act, V, dtype):  # noqa: F811
    """An infinite temperature draws evenly from what is not masked, as a huge one does; a tiny one is nearly greedy."""
    t, d, x, u, e = drafts(4, 3, V, seed=V, dtype=dtype)
    t = torch.where(t > 0, t, -torch.inf)
    d[1] = torch.where(d[1] > 0, d[1], -torch.inf)
    for extreme, plain in ((torch.inf, 1e30), (3e38, 1e30), (1e-45, 1e-20), (1e-38, 1e-20)):
        # (at 1e30 every difference of logits is 0 to fp32, at 1e-20 any that is not 0 takes the smaller one's weight)
        want = check_verify(fp8act, t, d, x, u, e, torch.full((4,), plain, device="cuda"))
        got = fp8act.verify_drafts(t, x, u, e, torch.full((4,), extreme, device="cuda"), draft_logits=d)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), extreme
        assert all(v >= 0 and t[b, int(got[0][b]), v] > -torch.inf
                   for b in range(4) for v in [int(got[1][b, int(got[0][b])])])


# ------------------------------------------------------------------ layout
@pytest.mark.parametrize("T", [0, 1])
def test_single_token_of_odd_rows(fp8act, T):  # noqa: F811
    """The distance to a next token that is not there does not matter."""
    H, D = 2, 128
    rows = randn(3, (2 + 2 + 4) * D + 3, seed=1)
    q, k, v = (rows[:, n:m].unflatten(1, (-1, D))[:T] for n, m in ((0, 4 * D), (4 * D, 6 * D), (6 * D, 8 * D)))
    assert T == 0 or q.stride(0) % 8
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens = torch.full((1,), T, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = []
    for a, b, c in ((q, k, v), (q.contiguous(), k.contiguous(), v.contiguous())):
        cache = fp8act.kv_cache(1, H, 16, D)
        fp8act.fp8_kv_append(b, c, torch.arange(T, device="cuda"), cache)
        out.append((fp8act.fp8_kv_attention(a, cache, table, lens, cu), *cache))
    assert all(torch.equal(a, b) for a, b in zip(*out))


# --------------------------------------------- verification: distribution
@pytest.mark.parametrize("temperature", [1.0, 0.6])
@pytest.mark.parametrize("greedy_draft", [False, True])
def test_verify_keeps_the_targets_distribution_in_many_draws(fp8act, greedy_draft, temperature):  # noqa: F811
    """960000 first tokens, chi-square over 6 tokens: below 35.9, which 5 degrees of freedom pass with 1 - 1e-6."""
    B, V, rounds = 60000, 6, 16
    t = torch.tensor([0.3, -1.0, 1.1, 0.0, -2.0, 0.6], device="cuda").expand(B, 2, V).contiguous()
    d = torch.tensor([1.0, 0.5, -0.5, 0.0, 0.2, 0.1], device="cuda").expand(B, 1, V).contiguous()
    temp = torch.full((B,), temperature, device="cuda")
    seen = torch.zeros(V, dtype=torch.float64, device="cuda")
    for i in range(rounds):
        g = gen(1000 + i)
        race = torch.empty((B, 1, V), device="cuda").exponential_(generator=g)
        x = ((d / temperature).softmax(-1) / race).argmax(-1).to(torch.int32)
        if greedy_draft:
            x = torch.full_like(x, 2)
        u = torch.rand((B, 1), device="cuda", generator=g)
        e = torch.empty((B, V), device="cuda").exponential_(generator=g)
        _, tokens, _ = fp8act.verify_drafts(t, x, u, e, temp, draft_logits=None if greedy_draft else d)
        seen += torch.bincount(tokens[:, 0].long(), minlength=V).double()
    want = (t[0, 0].double() / temperature).softmax(-1) * B * rounds
    assert float(((seen - want) ** 2 / want).sum()) < 35.9
