"""The operators around the cache reject bad arguments on the host (no kernel runs in these tests)."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch
from test_decoder_ops_abi import A16, ALIGN, DEVICE, NULL, OK, SHAPE, cache, lib  # noqa: F401

from block_scaled_fp8_act_gb300 import build as fp8build
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


def evict(lib, mass=A16, table=A16, mp=4, lens=A16, keep=A16 + 64, new=A16, np=2, B=1, recent=0, first=0, out=A16 + 128, kept=A16,  # noqa: F811
          c=None, **kw):
    return lib.fp8_kv_evict(ctypes.byref(cache(**kw)) if c is None else c, mass, table, mp, lens, keep, new, np, B, recent, first,
                            out, kept, None)


def test_evict_argument_checks(lib):  # noqa: F811
    for bad in (dict(page=24), dict(dim=96), dict(B=-1), dict(mp=-1), dict(np=-1), dict(recent=-1), dict(first=-1), dict(mp=1 << 26),
                dict(np=1 << 26), dict(B=1 << 30), dict(np=1 << 20, B=1 << 12), dict(pages=0), dict(out=A16), dict(out=A16 + 64)):
        assert evict(lib, **bad) == SHAPE, bad
    assert evict(lib, B=0, mass=None, lens=None) == OK
    for name in ("mass", "table", "lens", "keep", "new", "out", "kept"):
        assert evict(lib, **{name: None}) == NULL, name
    for bad in (dict(mass=A16 + 8), dict(table=A16 + 2), dict(lens=A16 + 1), dict(keep=A16 + 2), dict(new=A16 + 3), dict(out=A16 + 2),
                dict(kept=A16 + 2)):
        assert evict(lib, **bad) == ALIGN, bad
    if not torch.cuda.is_available():
        assert evict(lib) == DEVICE and evict(lib, np=0, new=None, kept=None) == DEVICE


def test_structs_match_the_header():
    text = open(os.path.join(fp8build.INCLUDE, "fp8act.h"), encoding="utf-8").read()
    body = re.search(r"typedef struct \{([^{}]*)\}\s*fp8act_scores;", text).group(1)
    assert re.findall(r"(\w+)(?:,|;)", body) == [f[0] for f in fp8act.ScoresStruct._fields_]
    assert ctypes.sizeof(fp8act.ScoresStruct) == 32


def scored(lib, mass, q=A16, qs=1024, cu=A16, lens=A16, table=A16, mp=4, B=1, T=1, mq=1, hq=8, scale=0.1, out=A16, lse=A16, ws=A16,  # noqa: F811
           old=None, cap=0.0, window=0, prefix=None, first=None, slopes=None, scores=True, **kw):
    s = ctypes.byref(fp8act.ScoresStruct(cap, window, prefix, first, slopes)) if scores else None
    c = ctypes.byref(cache(**kw))
    if mass:
        return lib.fp8_kv_attention_mass(q, qs, cu, lens, table, mp, B, T, mq, hq, scale, s, c, lse, out, 1, old, None)
    return lib.fp8_kv_attention_scored(q, qs, cu, lens, table, mp, B, T, mq, hq, scale, s, c, out, lse, ws, 1 << 40, None)


@pytest.mark.parametrize("mass", [False, True])
def test_score_argument_checks(lib, mass):  # noqa: F811
    inf, nan = float("inf"), float("nan")
    for bad in (dict(cap=-1.0), dict(cap=nan), dict(cap=inf), dict(cap=1e-32), dict(cap=1e31), dict(window=-1), dict(hq=7), dict(hq=0),
                dict(qs=1000), dict(B=-1), dict(T=-1), dict(mq=-1), dict(mp=-1), dict(mp=1 << 26), dict(hq=514, qs=1 << 20),
                dict(scale=0.0), dict(scale=nan), dict(pages=0), dict(page=48)):
        assert scored(lib, mass, **bad) == SHAPE, bad
    assert scored(lib, mass, B=0, q=None) == OK
    for name in ("q", "cu", "lens", "table", "out") + (("lse",) if mass else ("ws",)):
        assert scored(lib, mass, **{name: None}) == NULL, name
    for bad in (dict(prefix=A16 + 2), dict(first=A16 + 1), dict(slopes=A16 + 2), dict(q=A16 + 8), dict(qs=1028), dict(lse=A16 + 2),
                dict(out=A16 + 4), dict(lens=A16 + 2)) + ((dict(old=A16 + 2),) if mass else ()):
        assert scored(lib, mass, **bad) == ALIGN, bad
    if not torch.cuda.is_available():
        for ok in (dict(), dict(cap=30.0, window=5, prefix=A16, first=A16, slopes=A16), dict(scores=False)):
            assert scored(lib, mass, **ok) == DEVICE
