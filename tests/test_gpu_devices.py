"""Tensors of another device than the current one are refused on the host, each argument by itself: a stand-in that claims
to be on a second GPU and has no memory takes one tensor's place, so that a call that went on would have no pointer."""
from __future__ import annotations

import pytest
import torch
from test_gpu_decoder_ops import clean_status, fp8act, randn  # noqa: F401  (fixtures too)

pytestmark = pytest.mark.gpu


class Elsewhere(torch.Tensor):
    """A tensor of a second GPU that holds no memory."""
    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_wrapper_subclass(cls, t.shape, dtype=t.dtype, device=torch.device("cuda", t.device.index + 1))

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


def calls(fp8act):  # noqa: F811
    """(Function, its tensors, the rest) of every operator."""
    T, Hq, H, D, B, page = 3, 4, 2, 64, 2, 16
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    c = fp8act.kv_cache(4, H, page, D)
    cache = dict(k_codes=c.k, v_codes=c.v, k_scale=c.k_scale, v_scale=c.v_scale)
    q, k, v = randn(T, Hq, D, seed=1), randn(T, H, D, seed=2), randn(T, H, D, seed=3)
    slots = torch.full((T,), -1, device="cuda")
    rows = dict(q=q, page_table=i32([0], [1]), kv_lens=i32(5, 7), cu_q=i32(0, 1, 3))
    scores = dict(prefix_lens=i32(0, 0), first=i32(0, 0, 0), slopes=f32(Hq))
    x, res = randn(T, 128, seed=4), randn(T, 128, seed=5)
    yield fp8act.fp8_rmsnorm_quant, dict(x=x, weight=x[0].clone(), residual=res, q=u8(T, 128), sa=f32(T, 1),
                                         residual_out=torch.empty_like(x)), {}
    yield fp8act.fp8_silu_mul_quant, dict(gate_up=randn(T, 256, seed=6), q=u8(T, 128), sa=f32(T, 1)), {}
    yield fp8act.fp8_kv_append, dict(k=k, v=v, slots=slots, **cache), {}
    yield fp8act.fp8_rope_append, dict(q=q, k=k, v=v, positions=torch.zeros((1, T), dtype=torch.int64, device="cuda"),
                                       inv_freq=torch.ones(D // 2, dtype=torch.float64, device="cuda"), slots=slots,
                                       q_weight=q[0, 0].clone(), k_weight=q[0, 0].clone(), axes=i32(*[0] * (D // 2)),
                                       q_out=torch.empty_like(q), **cache), {}
    need = fp8act.kv_attention_workspace(2, Hq, c)
    yield fp8act.fp8_kv_attention, dict(out=torch.empty_like(q), lse=f32(T, Hq), workspace=u8(need), **rows, **scores, **cache), \
        dict(max_q_len=2)
    yield fp8act.fp8_kv_attention_mass, dict(lse=f32(T, Hq), mass=fp8act.kv_mass(c), old_lens=i32(4, 5), **rows, **scores, **cache), \
        dict(max_q_len=2)
    yield fp8act.fp8_kv_evict, dict(mass=fp8act.kv_mass(c), page_table=i32([0], [1]), kv_lens=i32(5, 7), keep=i32(2, 3),
                                    new_table=i32([2], [3]), new_lens=i32(0, 0), kept=torch.empty((B, H, page), dtype=torch.int32,
                                                                                               device="cuda"), **cache), {}
    yield fp8act.verify_drafts, dict(target_logits=f32(B, 2, 32), draft_tokens=i32([0], [1]), uniform=f32(B, 1), noise=f32(B, 32) + 1,
                                     temperature=f32(B) + 1, draft_logits=f32(B, 1, 32), n_draft=i32(1, 1), accepted=i32(0, 0),
                                     tokens=i32([0, 0], [0, 0]), accept_prob=f32(B, 1),
                                     workspace=u8(fp8act.verify_drafts_workspace(B, 1))), {}


def run(fp8act, function, tensors, rest):  # noqa: F811
    a = dict(tensors)
    if "k_codes" in a:
        a["cache"] = fp8act.KvCache(*(a.pop(n) for n in ("k_codes", "v_codes", "k_scale", "v_scale")))
    return function(**a, **rest)


def test_every_tensor_is_on_the_current_device(fp8act):  # noqa: F811
    n = 0
    for function, tensors, rest in calls(fp8act):
        run(fp8act, function, tensors, rest)
        for name, t in tensors.items():
            with pytest.raises(ValueError, match="not on the current CUDA device"):
                run(fp8act, function, {**tensors, name: Elsewhere(t)}, rest)
            n += 1
        run(fp8act, function, tensors, rest)
    assert n > 70
