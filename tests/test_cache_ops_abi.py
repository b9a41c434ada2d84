"""The operators around the cache reject bad arguments on the host (no kernel runs in these tests)."""
from __future__ import annotations

import ctypes

import pytest
import torch
from test_decoder_ops_abi import A16, ALIGN, DEVICE, NULL, OK, SHAPE, cache, lib  # noqa: F401

from block_scaled_fp8_act_gb300 import fp8act


def rope(lib, q=A16, k=A16, v=A16, qs=1024, ks=256, vs=256, qw=None, kw=None, pos=A16, freq=A16, axis=None, n_axes=1, rot=128,  # noqa: F811
         slots=A16, T=1, hq=8, out=A16, c=None, **kw2):
    return lib.fp8_rope_append(q, k, v, qs, ks, vs, qw, kw, 1e-6, 0.0, pos, freq, axis, n_axes, rot, 0, 1.0, slots, T, hq,
                               ctypes.byref(cache(**kw2)) if c is None else c, out, None)


def test_rope_argument_checks(lib):  # noqa: F811
    assert rope(lib, page=24) == SHAPE and rope(lib, dim=96) == SHAPE and rope(lib, heads=0) == SHAPE
    for bad in (dict(T=-1), dict(hq=0), dict(hq=1 << 21), dict(n_axes=0), dict(n_axes=5), dict(rot=-16), dict(rot=144),
                dict(rot=8), dict(rot=100), dict(qs=1016), dict(ks=248), dict(vs=128)):
        assert rope(lib, **bad) == SHAPE, bad
    assert rope(lib, T=0, q=None, k=None, v=None, pos=None, freq=None, slots=None, out=None) == OK
    for name in ("q", "k", "v", "pos", "freq", "slots", "out"):
        assert rope(lib, **{name: None}) == NULL, name
    for bad in (dict(q=A16 + 8), dict(k=A16 + 2), dict(v=A16 + 8), dict(qs=1028), dict(ks=260), dict(vs=258), dict(qw=A16 + 8),
                dict(kw=A16 + 4), dict(pos=A16 + 4), dict(freq=A16 + 4), dict(axis=A16 + 2), dict(slots=A16 + 4),
                dict(out=A16 + 8)):
        assert rope(lib, **bad) == ALIGN, bad
    if not torch.cuda.is_available():
        assert rope(lib) == DEVICE and rope(lib, rot=0, freq=None) == DEVICE


def test_binding_rejects_what_is_not_on_the_gpu(lib):  # noqa: F811
    c = (torch.zeros((1, 1, 16, 64), dtype=torch.uint8),) * 2 + (torch.zeros((1, 1, 16)),) * 2
    x, i = torch.zeros((1, 1, 64), dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(TypeError):
        fp8act.fp8_rope_append(x, x, x, i, torch.zeros(32, dtype=torch.float64), i, c)
