"""The paged cache's bookkeeping on the host: refused arguments, and the oracle
pinned by invariants.  CPU only: no call here launches a kernel."""
import numpy as np
import pytest

import mla_prefill_attention_plan_gb300 as mla
from mla_prefill_attention_plan_gb300 import build as B
from oracle import pages_oracle as P


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mla.load()


def _caller(fn, names, ok, **fixed):
    names = names.split()

    def call(**change):
        a, kw = list(ok), dict(fixed)
        for k, v in change.items():
            if k in names:
                a[names.index(k)] = v
            else:
                kw[k] = v
        return fn(*a, stream=1, **kw)   # any non-null handle: these calls fail before using it
    return call


@pytest.mark.parametrize("change", [
    dict(dt=None), dict(dl=None), dict(st=None), dict(sl=None), dict(rc=None), dict(par=None), dict(np=0), dict(mp=0),
    dict(db=-1), dict(sb=-1), dict(db=1 << 30, sb=1 << 30), dict(dt=1 << 20), dict(dt=(1 << 20) - 4 * 8 * 2 + 4),
    dict(dl=(1 << 21) + 4)])
def test_fork_refusals(lib, change):
    call = _caller(mla.mla_pages_fork, "dt dl st sl rc par np mp db sb",
                   [1 << 16, 1 << 17, 1 << 20, 1 << 21, 1 << 22, 1 << 23, 8, 8, 2, 3])
    assert call(**change) == mla.MLA_ERR_ARG


@pytest.mark.parametrize("change", [dict(pt=None), dict(rc=None), dict(cl=None), dict(np=0), dict(ps=0), dict(mp=0),
                                    dict(b=-1)])
def test_free_refusals(lib, change):
    call = _caller(mla.mla_pages_free, "pt rc cl keep np ps mp b", [16, 16, 16, None, 8, 16, 4, 2])
    assert call(**change) == mla.MLA_ERR_ARG


def test_workspace(lib):
    size = mla.mla_pages_workspace_bytes
    assert size(0, 4) == 0 and size(8, -1) == 0
    assert size(1000, 7) >= 4 * 4000 + 7 * 8 and size(1000, 7) % 256 == 0
    assert size(1 << 30, 1 << 20) >= 16 << 30


@pytest.mark.parametrize("change", [dict(pt=None), dict(rc=None), dict(cl=None), dict(new=None), dict(cs=None),
                                    dict(cd=None), dict(cc=None), dict(np=0), dict(ps=0), dict(mp=0), dict(b=-1)])
def test_reserve_refusals(lib, change):
    call = _caller(mla.mla_pages_reserve, "pt rc cl new cs cd cc np ps mp b",
                   [16, 16, 16, 16, 16, 16, 16, 8, 16, 4, 2], workspace=256, workspace_bytes=1 << 20)
    assert call(**change) == mla.MLA_ERR_ARG
    for ws in (dict(workspace=None), dict(workspace=128), dict(workspace_bytes=mla.mla_pages_workspace_bytes(8, 2) - 1)):
        assert call(**ws) == mla.MLA_ERR_WORKSPACE


@pytest.mark.parametrize("change", [dict(pt=None), dict(rc=None), dict(cs=None), dict(cd=None), dict(cc=None),
                                    dict(most=-1), dict(np=0), dict(mp=0), dict(b=-1)])
def test_compact_refusals(lib, change):
    call = _caller(mla.mla_pages_compact, "pt rc cs cd cc most np mp b", [16, 16, 16, 16, 16, 8, 8, 4, 2],
                   workspace=256, workspace_bytes=1 << 20)
    assert call(**change) == mla.MLA_ERR_ARG
    for ws in (dict(workspace=None), dict(workspace=128), dict(workspace_bytes=mla.mla_pages_workspace_bytes(8, 2) - 1)):
        assert call(**ws) == mla.MLA_ERR_WORKSPACE


@pytest.mark.parametrize("change", [dict(kv=None), dict(kv=18), dict(bytes=0), dict(bytes=6), dict(bytes=1 << 31),
                                    dict(layers=-1), dict(stride=64), dict(stride=130), dict(src=None), dict(dst=None),
                                    dict(cnt=None), dict(most=-1), dict(np=0)])
def test_copy_refusals(lib, change):
    call = _caller(mla.mla_pages_copy, "kv bytes layers stride src dst cnt most np", [16, 16, 2, 128, 16, 16, 16, 4, 8])
    assert call(**change) == mla.MLA_ERR_ARG


@pytest.mark.parametrize("change", [dict(kv=None), dict(kv=18), dict(bytes=0), dict(bytes=6), dict(layers=-1),
                                    dict(layers=65536), dict(stride=16), dict(stride=514), dict(cl=None),
                                    dict(keep=None), dict(ks=0), dict(kc=None), dict(pt=None), dict(np=0), dict(ps=0),
                                    dict(mp=0), dict(b=-1), dict(np=1 << 20, ps=1 << 11)])
def test_keep_rows_refusals(lib, change):
    call = _caller(mla.mla_cache_keep_rows, "kv bytes layers stride cl keep ks kc pt np ps mp b",
                   [16, 16, 2, 512, 16, 16, 4, 16, 16, 8, 4, 2, 2])
    assert call(**change) == mla.MLA_ERR_ARG


@pytest.mark.parametrize("change", [dict(rope=None), dict(kv=None), dict(kv=24), dict(lat=None), dict(gamma=20),
                                    dict(freqs=None), dict(iro=None), dict(cl=None), dict(pt=None), dict(np=0),
                                    dict(ps=0), dict(mp=0), dict(B=0), dict(H=0), dict(T=-1), dict(L=0),
                                    dict(eps=-1.0), dict(inv=0.0)])
def test_write_at_refusals(lib, change):
    call = _caller(mla.mla_latent_cache_write_at, "kv q lat gamma freqs rope iro cl pt np ps mp B H T L eps inv dt",
                   [16, 16, 16, 16, 16, 16, 16, 16, 16, 4, 16, 2, 1, 2, 8, 64, 1e-6, 1.0, mla.MLA_BF16])
    assert call(**change) == mla.MLA_ERR_ARG
    assert call(dt=7) == mla.MLA_ERR_DTYPE


def test_status_text(lib):
    assert "free pages" in mla.status_string(mla.MLA_DEV_NO_PAGES)


# ------------------------------------------------------------------ the oracle

def consistent(table, refs):
    held = np.bincount(table[table >= 0], minlength=len(refs))
    return np.array_equal(held, refs)


def walk(seed, steps=60):
    """A pool under random calls; every cache row carries the token it is for."""
    rng = np.random.default_rng(seed)
    B, page, pool, most = 6, 4, 60, 10
    table, refs, lengths = np.full((B, most), -1, np.int32), np.zeros(pool, np.int32), np.zeros(B, np.int64)
    cache, text, word = np.full((1, pool * page), -1), [[] for _ in range(B)], 0
    for _ in range(steps):
        op = rng.integers(4)
        if op == 0:
            parents = rng.integers(-1, B, B)
            table, lengths = P.fork(table, lengths, refs, parents)
            text = [list(text[p]) if p >= 0 else [] for p in parents]
        elif op == 1:
            keep = rng.integers(0, page * most, B)
            P.free(table, refs, lengths, keep, page)
            text = [t[:int(n)] for t, n in zip(text, lengths)]
        elif op == 2:
            moves = P.compact(table, refs, int(rng.integers(0, 20)))
            P.copy(cache.reshape(1, pool, page), moves)
        else:
            new = np.minimum(rng.integers(0, 9, B), page * most - lengths)
            before = table.copy(), refs.copy()
            copies = P.reserve(table, refs, lengths, new, page)
            if copies is None:
                assert np.array_equal(before[0], table) and np.array_equal(before[1], refs)
                continue
            P.copy(cache.reshape(1, pool, page), copies)
            for b in range(B):
                for _ in range(new[b]):
                    p = int(lengths[b])
                    cache[0, table[b, p // page] * page + p % page] = word
                    text[b].append(word)
                    word, lengths[b] = word + 1, p + 1
        assert consistent(table, refs)
        for b in range(B):
            at = np.arange(len(text[b]))
            assert list(cache[0, table[b, at // page] * page + at % page]) == text[b]


@pytest.mark.parametrize("seed", range(20))
def test_oracle_keeps_every_sequences_rows(seed):
    walk(seed)


def test_oracle_last_holder_keeps_the_page():
    table, refs = np.array([[3, -1], [3, -1], [3, -1]], np.int32), np.array([0, 0, 0, 3], np.int32)
    assert P.reserve(table, refs, np.array([5, 5, 5]), np.array([1, 1, 1]), 8) == [(3, 0), (3, 1)]
    assert table[:, 0].tolist() == [0, 1, 3] and refs.tolist() == [1, 1, 0, 1]


def test_oracle_compact_ends_dense():
    rng = np.random.default_rng(3)
    refs = (rng.random(50) < 0.4).astype(np.int32) * rng.integers(1, 4, 50).astype(np.int32)
    table = np.repeat(np.arange(50), refs).reshape(1, -1).astype(np.int32)
    total, n = sorted(refs), int((refs > 0).sum())
    P.compact(table, refs, 1 << 30)
    assert (refs[:n] > 0).all() and not refs[n:].any() and sorted(refs) == total and consistent(table, refs)


def test_oracle_keep_rows():
    cache = np.arange(32)[None].copy()
    P.keep_rows(cache, [5], [[0, 2, 3, 6]], np.array([[1, 0, 3]]), 8)
    # positions 5, 6, 7, 8 become what 5, 7, 8, 11 were: rows 13, 15, 0, 3
    assert cache[0, [13, 14, 15, 0]].tolist() == [13, 15, 0, 3]


HUGE = (1 << 31) - 65535       # one more than a count may be: the kernels' loops step past their ends


def test_sizes_that_32_bits_are_too_few_for(lib):
    fork = _caller(mla.mla_pages_fork, "dt dl st sl rc par np mp db sb",
                   [1 << 16, 1 << 17, 1 << 50, 1 << 51, 1 << 22, 1 << 23, 8, 8, 2, 3])
    free = _caller(mla.mla_pages_free, "pt rc cl keep np ps mp b", [16, 16, 16, None, 8, 16, 4, 2])
    reserve = _caller(mla.mla_pages_reserve, "pt rc cl new cs cd cc np ps mp b",
                      [16, 16, 16, 16, 16, 16, 16, 8, 16, 4, 2], workspace=256, workspace_bytes=1 << 50)
    compact = _caller(mla.mla_pages_compact, "pt rc cs cd cc most np mp b", [16, 16, 16, 16, 16, 8, 8, 4, 2],
                      workspace=256, workspace_bytes=1 << 50)
    keep = _caller(mla.mla_cache_keep_rows, "kv bytes layers stride cl keep ks kc pt np ps mp b",
                   [16, 16, 2, 512, 16, 16, 4, 16, 16, 8, 4, 2, 2])
    for call, names in ((fork, "np mp db sb"), (free, "np mp b"), (reserve, "np mp b"), (compact, "most np mp b"),
                        (keep, "ks b")):
        for name in names.split():
            for size in (HUGE, (1 << 31) - 1):
                assert call(**{name: size}) == mla.MLA_ERR_ARG, (call, name)
    assert reserve(mp=1 << 20, b=1 << 11) == mla.MLA_ERR_ARG         # entries, and so the pages that may be wanted
    assert mla.mla_pages_workspace_bytes(HUGE, 1) == 0 and mla.mla_pages_workspace_bytes(1, HUGE) == 0
    assert mla.mla_pages_workspace_bytes(HUGE - 1, HUGE - 1) > 0
