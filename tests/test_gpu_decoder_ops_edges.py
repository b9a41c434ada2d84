"""GPU tests of the operators between the linear layers where a caller's memory,
streams or values are unusual: views at odd offsets, streams that are passed,
producers right in front, ends of the number range."""
from __future__ import annotations

import pytest
import torch
from test_gpu_decoder_ops import check_verify, clean_status, drafts, fp8act, gen  # noqa: F401  (fixtures among them)

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
