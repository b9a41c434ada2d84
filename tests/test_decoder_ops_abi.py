"""The operators between the linear layers reject bad arguments on the host
(no kernel runs in these tests)."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from block_scaled_fp8_act_gb300 import build as fp8build
from block_scaled_fp8_act_gb300 import fp8act

OK, NULL, SHAPE, ALIGN, LAUNCH, TIMEOUT, DEVICE, CUDA, INDEX = range(9)
A16 = 0x10000  # a fake aligned address: never dereferenced, the checks run first


@pytest.fixture(scope="module")
def lib():
    fp8build.build()
    return fp8act.load()


def cache(**kw):
    d = dict(k=A16, v=A16, ks=A16, vs=A16, pages=4, page=64, heads=2, dim=128)
    d.update(kw)
    return fp8act.KvCacheStruct(d["k"], d["v"], d["ks"], d["vs"], d["pages"], d["page"], d["heads"], d["dim"])


def test_new_symbols_and_status(lib):
    names = set(fp8act.header_symbols())
    assert {"fp8_rmsnorm_quant", "fp8_silu_mul_quant", "fp8_kv_append", "fp8_kv_attention",
            "fp8_kv_attention_workspace", "fp8act_verify_drafts"} <= names
    assert "index" in fp8act.strerror(INDEX)
    assert fp8act.STATUS[INDEX] == "FP8ACT_ERR_INDEX"


def test_cache_struct_matches_the_header():
    text = open(os.path.join(fp8build.INCLUDE, "fp8act.h"), encoding="utf-8").read()
    body = re.search(r"typedef struct \{([^{}]*)\}\s*fp8act_kv_cache;", text).group(1)
    assert re.findall(r"(\w+)(?:,|;)", body) == [f[0] for f in fp8act.KvCacheStruct._fields_]
    assert ctypes.sizeof(fp8act.KvCacheStruct) == 48


def test_rmsnorm_argument_checks(lib):
    f = lib.fp8_rmsnorm_quant
    call = lambda x=A16, r=A16, w=A16, M=1, K=128, q=A16, sa=A16, o=A16: f(x, r, w, 1e-6, 0.0, M, K, q, sa, o, None)  # noqa: E731
    assert call(K=100) == SHAPE and call(K=0) == SHAPE and call(M=-1) == SHAPE and call(K=32896) == SHAPE
    assert call(x=None, r=None, w=None, M=0, q=None, sa=None, o=None) == OK
    assert call(x=None) == NULL and call(w=None) == NULL and call(q=None) == NULL and call(sa=None) == NULL
    assert call(r=None) == NULL and call(o=None) == NULL           # residual without its output, and the reverse
    assert call(x=A16 + 8) == ALIGN and call(r=A16 + 2) == ALIGN and call(w=A16 + 8) == ALIGN
    assert call(q=A16 + 4) == ALIGN and call(o=A16 + 4) == ALIGN and call(sa=A16 + 2) == ALIGN


def test_silu_argument_checks(lib):
    f = lib.fp8_silu_mul_quant
    assert f(A16, 1, 64, A16, A16, None) == SHAPE
    assert f(A16, -1, 128, A16, A16, None) == SHAPE
    assert f(None, 0, 128, None, None, None) == OK
    assert f(None, 1, 128, A16, A16, None) == NULL
    assert f(A16 + 8, 1, 128, A16, A16, None) == ALIGN
    assert f(A16, 1, 128, A16 + 8, A16, None) == ALIGN


def test_append_argument_checks(lib):
    f = lib.fp8_kv_append

    def call(k=A16, v=A16, s=A16, T=1, ks=256, vs=256, c=None, **kw):
        return f(k, v, s, T, ks, vs, ctypes.byref(cache(**kw)) if c is None else c, None)
    assert f(A16, A16, A16, 1, 256, 256, None, None) == NULL
    for bad in (dict(page=8), dict(page=48), dict(page=512), dict(dim=96), dict(dim=512), dict(heads=0), dict(pages=-1)):
        assert call(**bad) == SHAPE, bad
    assert call(T=-1) == SHAPE and call(ks=255) == SHAPE and call(vs=128) == SHAPE
    assert call(k=None, v=None, s=None, T=0) == OK
    assert call(k=None) == NULL and call(v=None) == NULL and call(s=None) == NULL
    for which in ("k", "v", "ks", "vs"):
        assert f(A16, A16, A16, 1, 256, 256, ctypes.byref(cache(**{which: None})), None) == NULL
        assert f(A16, A16, A16, 1, 256, 256, ctypes.byref(cache(**{which: A16 + 8})), None) == ALIGN
    assert call(k=A16 + 8) == ALIGN and call(ks=260) == ALIGN and call(s=A16 + 4) == ALIGN


def test_attention_argument_checks(lib):
    f, size = lib.fp8_kv_attention, lib.fp8_kv_attention_workspace
    c = cache()
    need = size(1, 8, ctypes.byref(c))
    assert need > 0 and size(8, 8, ctypes.byref(c)) > need
    assert size(1, 7, ctypes.byref(c)) == 0 and size(-1, 8, ctypes.byref(c)) == 0
    assert size(1, 8, ctypes.byref(cache(dim=80))) == 0 and size(1, 8, None) == 0

    def call(q=A16, qs=1024, cu=A16, lens=A16, table=A16, mp=4, B=1, T=1, mq=1, hq=8, out=A16, lse=None, ws=A16,
             n=1 << 40, cc=None):
        return f(q, qs, cu, lens, table, mp, B, T, mq, hq, 0.1, ctypes.byref(cc or c), out, lse, ws, n, None)
    assert call(hq=7) == SHAPE and call(hq=0) == SHAPE and call(qs=1000) == SHAPE and call(B=-1) == SHAPE
    assert call(T=-1) == SHAPE and call(mq=-1) == SHAPE and call(mp=-1) == SHAPE and call(mp=1 << 26) == SHAPE
    assert call(hq=2 * 257, qs=1 << 20) == SHAPE
    assert call(n=need - 1) == SHAPE
    assert call(B=0) == OK and call(q=None, cu=None, T=0) == OK
    for name in ("q", "cu", "lens", "table", "out", "ws"):
        assert call(**{name: None}) == NULL, name
    assert call(q=A16 + 8) == ALIGN and call(qs=1028) == ALIGN and call(out=A16 + 4) == ALIGN
    assert call(ws=A16 + 4) == ALIGN and call(lens=A16 + 2) == ALIGN and call(lse=A16 + 1) == ALIGN


def test_verify_argument_checks(lib):
    f = lib.fp8act_verify_drafts

    def call(t=A16, d=A16, f32=0, x=A16, u=A16, e=A16, temp=A16, n=None, B=1, k=2, V=100, a=A16, out=A16, pr=None,
             ws=A16, size=1 << 40):
        return f(t, d, f32, x, u, e, temp, n, B, k, V, a, out, pr, ws, size, None)
    need = lib.fp8act_verify_drafts_workspace(1, 2)
    assert 0 < need < lib.fp8act_verify_drafts_workspace(34, 2)
    assert lib.fp8act_verify_drafts_workspace(1, 33) == 0 and lib.fp8act_verify_drafts_workspace(-1, 2) == 0
    assert call(size=need - 1) == SHAPE and call(B=65536) == SHAPE and call(ws=A16 + 4) == ALIGN
    assert call(k=33) == SHAPE and call(k=-1) == SHAPE and call(V=0) == SHAPE and call(B=-1) == SHAPE
    assert call(t=None, B=0) == OK
    for name in ("t", "x", "u", "e", "temp", "a", "out", "ws"):
        assert call(**{name: None}) == NULL, name
    assert call(t=A16 + 2) == ALIGN and call(d=A16 + 8) == ALIGN and call(e=A16 + 2) == ALIGN
    assert call(pr=A16 + 1) == ALIGN


def test_binding_rejects_what_is_not_on_the_gpu():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fp8act.fp8_rmsnorm_quant(x, w)
    with pytest.raises(TypeError):
        fp8act.fp8_silu_mul_quant(torch.zeros((1, 256), dtype=torch.bfloat16))
    c = (torch.zeros((1, 1, 16, 64), dtype=torch.uint8),) * 2 + (torch.zeros((1, 1, 16)),) * 2
    with pytest.raises(TypeError):
        kv = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
        fp8act.fp8_kv_append(kv, kv, torch.zeros(1, dtype=torch.int64), c)


def test_a_call_without_a_gb300_is_refused(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    c = cache()
    assert lib.fp8_rmsnorm_quant(A16, None, A16, 1e-6, 0.0, 1, 128, A16, A16, None, None) == DEVICE
    assert lib.fp8_silu_mul_quant(A16, 1, 128, A16, A16, None) == DEVICE
    assert lib.fp8_kv_append(A16, A16, A16, 1, 256, 256, ctypes.byref(c), None) == DEVICE
    assert lib.fp8_kv_attention(A16, 1024, A16, A16, A16, 4, 1, 1, 1, 8, 0.1, ctypes.byref(c), A16, None, A16, 1 << 40,
                                None) == DEVICE
    assert lib.fp8act_verify_drafts(A16, None, 0, A16, A16, A16, A16, None, 1, 2, 100, A16, A16, None, A16, 1 << 40,
                                    None) == DEVICE
