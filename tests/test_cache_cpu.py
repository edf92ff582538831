"""Paged history cache and tree scorer without a GPU: the library's exports, and the calls it
refuses before any launch."""
import ctypes as C
import os
import re

import pytest
import torch

from conftest import ROOT

capi = pytest.importorskip("hstu_jagged_pointwise_b200.capi")
ops = pytest.importorskip("hstu_jagged_pointwise_b200.ops")
BAD, UNSUP, WS = capi.HSTU_ERR_INVALID_ARG, capi.HSTU_ERR_UNSUPPORTED, capi.HSTU_ERR_WORKSPACE
L = capi.CACHE
_mem = (C.c_uint8 * (1 << 20))()
BASE = (C.addressof(_mem) + 255) // 256 * 256          # any aligned address: nothing is launched


def test_exports_match_header():
    src = open(os.path.join(ROOT, "include", "hstu_cache.h")).read()
    names = set(re.findall(r"HSTU_API\s+[\w\s\*]+?\b(hstu_\w+)\s*\(", src))
    assert names == set(capi.CACHE_EXPORTS)
    out = os.popen(f"nm -D --defined-only {capi.CACHE_LIB_PATH}").read().split("\n")
    assert {l.split()[-1] for l in out if " T " in l} == names


def test_status_string_of_a_full_pool():
    assert capi.status_string(capi.HSTU_ERR_CACHE_FULL) != "unknown status"


def cache(**kw):
    base = dict(n_pages=8, page_size=16, n_slots=4, max_pages=4, row_elems=128, dtype=capi.HSTU_BF16, k=BASE, v=BASE, ts=BASE,
                page_table=BASE, lens=BASE, ref=BASE)
    base.update(kw)
    return capi.HstuPageCache(**base)


@pytest.mark.parametrize("kw,st", [
    (dict(n_pages=-1), BAD), (dict(n_slots=-1), BAD), (dict(max_pages=0), BAD), (dict(row_elems=0), BAD), (dict(dtype=5), BAD),
    (dict(page_size=0), UNSUP), (dict(page_size=24), UNSUP), (dict(page_size=256), UNSUP), (dict(row_elems=12), UNSUP),
    (dict(row_elems=6, dtype=capi.HSTU_F32), UNSUP), (dict(n_pages=1 << 28, page_size=128), UNSUP),
    (dict(max_pages=1 << 20), UNSUP), (dict(k=None), BAD), (dict(v=BASE + 8), BAD), (dict(ts=BASE + 4), BAD),
    (dict(page_table=None), BAD), (dict(lens=BASE + 2), BAD), (dict(ref=None), BAD)])
def test_cache_description_is_checked(kw, st):
    c = cache(**kw)
    assert L.hstu_cache_workspace_bytes(C.byref(c)) == 0
    assert L.hstu_cache_free(C.byref(c), 1, BASE, BASE, 1 << 20, None) == st
    assert L.hstu_cache_fork(C.byref(c), 1, BASE, BASE, BASE, 1 << 20, None) == st


def test_page_operators_refuse_before_launch():
    c = cache()
    need = L.hstu_cache_workspace_bytes(C.byref(c))
    assert need > 0 and need % 256 == 0
    r = C.byref(c)
    for fn, args in (("free", [BASE]), ("fork", [BASE, BASE]), ("append", [BASE, BASE, 0, None, 0, None, None, None]),
                     ("compact", [BASE, BASE, 0, None])):
        f = getattr(L, "hstu_cache_" + fn)
        assert f(None, 1, *args, BASE, need, None) == BAD
        assert f(r, -1, *args, BASE, need, None) == BAD
        assert f(r, 5, *args, BASE, need, None) == BAD                 # more requests than slots
        assert f(r, 1, *args, None, need, None) == WS
        assert f(r, 1, *args, BASE + 16, need, None) == WS
        assert f(r, 1, *args, BASE, need - 1, None) == WS
        assert f(r, 1, None, *args[1:], BASE, need, None) == BAD
        assert f(r, 0, *args, BASE, need, None) == capi.HSTU_OK
    a = lambda n=1, off=BASE, T=2, rows=None, n_src=2, k=BASE, v=BASE, ts=BASE: L.hstu_cache_append(
        r, n, BASE, off, T, rows, n_src, k, v, ts, BASE, need, None)
    assert a(T=-1) == BAD and a(n_src=1) == BAD and a(n_src=-1, rows=BASE) == BAD and a(n=0) == BAD
    assert a(off=None) == BAD and a(k=None) == BAD and a(v=BASE + 8) == BAD and a(ts=BASE + 4) == BAD and a(rows=BASE + 2) == BAD
    k = lambda n=1, off=BASE, K=2, rows=BASE: L.hstu_cache_compact(r, n, BASE, off, K, rows, BASE, need, None)
    assert k(K=-1) == BAD and k(n=0) == BAD and k(off=None) == BAD and k(rows=None) == BAD
    assert L.hstu_cache_check_device_error(BASE + 8, None) == WS
    assert L.hstu_cache_debug_set_wait_fault(-1, 0) == BAD and L.hstu_cache_debug_set_wait_fault(0, 2) == BAD


def tree(**kw):
    base = dict(B=2, T=6, H=2, d=64, n_pos=256, n_tbuckets=64, max_nodes=4, alpha=5.0, ln_eps=1e-5)
    base.update(kw)
    return capi.HstuTreeDims(**base)


@pytest.mark.parametrize("kw,ckw,st", [
    (dict(B=-1), {}, BAD), (dict(T=-1), {}, BAD), (dict(H=0), {}, BAD), (dict(B=0), {}, BAD), (dict(max_nodes=0), {}, BAD),
    (dict(alpha=0.0), {}, BAD), (dict(alpha=float("inf")), {}, BAD), (dict(ln_eps=-1.0), {}, BAD),
    (dict(ln_eps=float("nan")), {}, BAD), (dict(H=1), {}, BAD), (dict(d=32, H=4), {}, UNSUP), (dict(max_nodes=8193), {}, UNSUP),
    (dict(n_pos=0), {}, UNSUP), (dict(n_pos=1025), {}, UNSUP), (dict(n_tbuckets=65), {}, UNSUP),
    ({}, dict(dtype=capi.HSTU_F32), UNSUP), (dict(H=65, d=128), dict(row_elems=65 * 128), UNSUP), ({}, dict(page_size=8), UNSUP)])
def test_tree_sizes_are_checked(kw, ckw, st):
    d, c = tree(**kw), cache(**ckw)
    assert L.hstu_tree_workspace_bytes(C.byref(d), C.byref(c)) == 0
    assert L.hstu_tree_score(C.byref(d), C.byref(c), *[BASE] * 17, 1 << 20, None) == st


def test_tree_pointers_are_checked():
    d, c = tree(), cache()
    need = L.hstu_tree_workspace_bytes(C.byref(d), C.byref(c))
    assert need > 0
    call = lambda args, ws=BASE, n=need: L.hstu_tree_score(C.byref(d), C.byref(c), *args, ws, n, None)
    full = [BASE] * 16
    assert L.hstu_tree_score(None, C.byref(c), *full, BASE, need, None) == BAD
    assert L.hstu_tree_score(C.byref(d), None, *full, BASE, need, None) == BAD
    assert call(full, None) == WS and call(full, BASE, need - 1) == WS and call(full, BASE + 64) == WS
    for i in range(16):                                # each pointer missing, and off its alignment
        for bad in (None, BASE + 2):
            args = list(full)
            args[i] = bad
            assert call(args) == BAD, (i, bad)
    d0 = tree(B=0, T=0, max_nodes=0)
    n0 = L.hstu_tree_workspace_bytes(C.byref(d0), C.byref(c))
    assert L.hstu_tree_score(C.byref(d0), C.byref(c), *[None] * 16, BASE, n0, None) == capi.HSTU_OK


def test_python_refusals():
    with pytest.raises(ValueError):
        ops.PagedCache(4, 16, 2, 2, 128, torch.float16)
    with pytest.raises(ValueError):
        ops.PagedCache(4, 16, 2, 2, 128, torch.bfloat16, device="cpu")
