"""The cache-page operators without a GPU: the library exports what
include/pa_pages.h declares and refuses bad calls on the host, and the
oracle the GPU tests compare with keeps the invariants of a page pool."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import pages_oracle as O
from paged_latent_attention_cache_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    build.build()
    from paged_latent_attention_cache_gb300 import binding
    return binding


def _params(B, **kw):
    base = dict(num_blocks=32, block_size=16, max_blocks_per_seq=4, num_seqs=8)
    base.update(kw)
    return B.make_pages_params(**base)


def test_exports_match_header(B):
    src = open(os.path.join(ROOT, "include", "pa_pages.h")).read()
    declared = sorted(set(re.findall(r"\b(pa_pages_\w+)\s*\(", src)))
    assert declared == sorted(B.EXPORTED_PAGES)
    for name in declared:
        assert hasattr(B.lib, name)


@pytest.mark.parametrize("kw,needle", [
    (dict(num_blocks=0), "num_blocks"), (dict(num_blocks=(1 << 22) + 1), "num_blocks"),
    (dict(num_blocks=1 << 22, block_size=1024), "slot range"),
    (dict(block_size=24), "power of two"), (dict(block_size=8), "power of two"),
    (dict(max_blocks_per_seq=0), "max_blocks_per_seq"),
    (dict(max_blocks_per_seq=1 << 27, block_size=16), "int32"),
    (dict(num_seqs=0), "num_seqs"), (dict(num_seqs=(1 << 22) + 1), "num_seqs"),
])
def test_params_refused(B, kw, needle):
    p = _params(B, **kw)
    assert B.pa_pages_validate(p) == B.PA_ERR_INVALID_ARGUMENT
    assert needle in B.last_error()
    assert B.pa_pages_workspace_size(p) == 0


def _caches(B, n=1, data=0x10000, page_bytes=16 * 384):
    arr = (B.pa_pages_cache * max(n, 1))()
    for i in range(n):
        arr[i].data, arr[i].page_bytes = data, page_bytes
    return arr


def _vp(x):
    return ctypes.c_void_p(x) if x else None


def _all_calls(B, p, caches, nc, n=4, ws=0x200000, wsb=1 << 30, a=0x20000, b=0x30000, err=0x90000):
    """Every call that takes caches and a workspace, with fake pointers."""
    P = ctypes.byref(p)
    sz = ctypes.c_size_t(wsb)
    yield B.lib.pa_pages_copy(P, caches, nc, _vp(a), _vp(b), None, n, _vp(ws), sz, _vp(err), None)
    yield B.lib.pa_pages_fork(P, caches, nc, _vp(a), _vp(b), n, _vp(0x40000), _vp(0x50000),
                              _vp(0x60000), _vp(ws), sz, _vp(err), None)
    yield B.lib.pa_pages_compact(P, caches, nc, _vp(a), _vp(b), None, _vp(ws), sz, _vp(err), None)


@pytest.mark.parametrize("cache,nc,needle", [
    (dict(data=0x10008), 1, "16-byte"), (dict(data=0), 1, "16-byte"),
    (dict(page_bytes=16 * 24), 1, "page_bytes"), (dict(page_bytes=0), 1, "page_bytes"),
    (dict(page_bytes=-256), 1, "page_bytes"), ({}, -1, "num_caches"),
])
def test_caches_refused(B, cache, nc, needle):
    p = _params(B)
    for s in _all_calls(B, p, _caches(B, 1, **cache), nc):
        assert s == B.PA_ERR_INVALID_ARGUMENT and needle in B.last_error()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(a=0), 1, "NULL"), (dict(b=0), 1, "NULL"), (dict(a=0x20002), 1, "4-byte"),
    (dict(err=0x90002), 1, "4-byte"), (dict(ws=0x200010), 1, "256-byte"),
    (dict(ws=0), 4, "workspace"), (dict(wsb=64), 4, "workspace"),
])
def test_pointers_refused(B, kw, status, needle):
    for s in _all_calls(B, _params(B), _caches(B), 1, **kw):
        assert s == status, B.last_error()
        assert needle in B.last_error()


def test_counts_refused(B):
    P, c = ctypes.byref(_params(B)), _caches(B)
    sz = ctypes.c_size_t(1 << 30)
    v = _vp(0x20000)
    for n in (-1, 33):
        assert B.lib.pa_pages_copy(P, c, 1, v, v, None, n, v, sz, v, None) == 1
    for n in (-1, 9):
        assert B.lib.pa_pages_fork(P, c, 1, v, v, n, v, v, v, v, sz, v, None) == 1
        assert B.lib.pa_pages_free(P, v, n, v, v, v, v, None) == 1
    for t in (-1, 1 << 31):
        assert B.lib.pa_pages_reserve(P, v, t, v, v, v, v, v, sz, v, None) == 1
    assert B.lib.pa_pages_free(P, None, 2, v, v, v, v, None) == 1
    assert B.lib.pa_pages_reserve(P, None, 4, v, v, v, v, v, sz, v, None) == 1
    # nothing to do
    assert B.lib.pa_pages_copy(P, c, 1, v, v, None, 0, v, sz, v, None) == 0
    assert B.lib.pa_pages_fork(P, c, 1, v, v, 0, v, v, v, v, sz, v, None) == 0
    assert B.lib.pa_pages_free(P, v, 0, v, v, v, v, None) == 0
    assert B.lib.pa_pages_reserve(P, v, 0, v, v, v, v, v, sz, v, None) == 0


# ---- the oracle

def _pool(seed, ns=6, mb=5, nb=24, bs=16):
    rng = np.random.default_rng(seed)
    table = np.full((ns, mb), -1, np.int32)
    past, ref = np.zeros(ns, np.int32), np.zeros(nb, np.int32)
    cache = rng.integers(0, 1000, size=(nb, bs, 2)).astype(np.int32)
    return rng, [cache], table, past, ref


def _sound(table, past, ref, bs):
    named = np.bincount(table[table >= 0], minlength=len(ref))
    assert (named == ref).all()
    for b in range(len(past)):
        assert (table[b, :-(-int(past[b]) // bs)] >= 0).all()


@pytest.mark.parametrize("seed", range(20))
def test_oracle_keeps_a_sound_pool(seed):
    """Random reserve / fork / free / compact sequences: refcounts equal the
    entries that name a page, held positions have pages, and what a sequence
    reads through its table changes only where it wrote."""
    rng, caches, table, past, ref = _pool(seed)
    bs = 16
    view = {}  # sequence -> the rows it has to read
    for _ in range(40):
        what = rng.integers(4)
        if what == 0:
            q = rng.integers(0, 30, size=len(past))
            cum = np.concatenate([[0], np.cumsum(q)])
            err, slots = O.reserve(table, past, ref, cum, int(cum[-1]), bs)
            for b in range(len(past)):
                mine = slots[cum[b]:cum[b + 1]]
                if (mine < 0).any():
                    assert (mine < 0).all() and err
                    continue
                rows = rng.integers(0, 1000, size=(len(mine), 2))
                caches[0].reshape(-1, 2)[mine] = rows
                view[b] = np.concatenate([view.get(b, np.zeros((0, 2), int)), rows])
                past[b] += len(mine)
        elif what == 1:
            p, c = rng.integers(len(past)), rng.integers(len(past))
            err = O.fork(caches, table, past, ref, [p], [c], bs)
            if not err:
                view[c] = view.get(p, np.zeros((0, 2), int)).copy()
        elif what == 2:
            s = rng.integers(len(past))
            assert O.free(table, past, ref, [s, s]) == 0
            view[s] = np.zeros((0, 2), int)
        else:
            err, live = O.compact(caches, table, ref)
            assert err == 0 and (ref[:live] > 0).all() and (ref[live:] == 0).all()
        _sound(table, past, ref, bs)
        for b, rows in view.items():
            pos = np.arange(past[b])
            got = caches[0][table[b, pos // bs], pos % bs] if len(pos) else np.zeros((0, 2), int)
            assert (got == rows).all()
