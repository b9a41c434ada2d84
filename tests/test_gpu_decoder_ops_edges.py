"""GPU tests of the operators between the linear layers where a caller's memory,
streams or values are unusual: views at odd offsets, streams that are passed,
producers right in front, ends of the number range."""
from __future__ import annotations

import pytest
import torch
from test_gpu_decoder_ops import check_verify, clean_status, drafts, fp8act, gen, randn  # noqa: F401  (fixtures too)

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
