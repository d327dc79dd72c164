"""Eviction of the same sequences again and again, without a GPU: the oracle's pins and the
refusals of mita_cache_evict_aged (nothing here launches)."""
import ctypes

import numpy as np
import pytest
import torch

import compressed_attention_adaptive_gb300 as mita
from compressed_attention_adaptive_gb300 import build as mita_build
from oracle import cache as ocache

A = 1 << 20  # an address, never read


@pytest.fixture(scope="module")
def lib():
    mita_build.build()
    return mita.lib()


def _p(**kw):
    base = dict(B=2, H=8, H_kv=2, T=1, d=128, page=64, n_pages=10, max_pages=4)
    base.update(kw)
    return mita.CacheParams(**base)


def _evict(lib, p, cache=2 * A, table=3 * A, lens=4 * A, keep=5 * A, first=0, recent=0, acc=6 * A, age=11 * A, len_out=7 * A,
           out=8 * A, src=9 * A, ws=10 * A, n=1 << 19):
    x = lambda a: None if a is None else ctypes.c_void_p(a)
    return lib.mita_cache_evict_aged(p.ref, x(cache), x(table), x(lens), x(keep), first, recent, x(acc), x(age), x(len_out),
                                     x(out), x(src), x(ws), n, None)


def test_aged_pointers(lib):
    p = _p()
    for kw in (dict(age=None), dict(age=11 * A + 2), dict(age=2 * A), dict(age=3 * A + 4), dict(age=4 * A), dict(age=5 * A),
               dict(age=6 * A), dict(age=6 * A + 64), dict(age=7 * A), dict(age=8 * A), dict(age=8 * A - 4), dict(age=9 * A),
               dict(cache=None), dict(keep=None), dict(recent=-1), dict(len_out=5 * A), dict(src=6 * A)):
        assert _evict(lib, p, **kw) == 1, kw
        assert lib.mita_last_error()
    for kw in (dict(ws=None), dict(ws=10 * A + 8), dict(n=0), dict(src=None, n=0), dict(len_out=4 * A, out=6 * A, n=0)):
        assert _evict(lib, p, **kw) == 3, kw
    assert _evict(lib, _p(d=96)) == 2


def test_aged_binding(lib):
    p = _p()
    cache, lens = torch.zeros(p.pool_bytes, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    table, acc, ws = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 2, 256), torch.zeros(4096, dtype=torch.uint8)
    age = torch.zeros(2, 2, 256, dtype=torch.int32)
    for bad in (age, age.long(), age[:1], age[..., :255], acc):
        with pytest.raises(ValueError):
            mita.mita_cache_evict(p, cache, table, lens, lens.clone(), acc, ws, age=bad)


def test_in_order_births_are_places():
    rng = np.random.default_rng(0)
    for n, keep, first, recent in ((50, 20, 3, 5), (50, 50, 1, 2), (7, 9, 0, 3), (30, 8, 3, 5), (300, 299, 0, 17)):
        acc = rng.integers(0, 5, n).astype(float)
        assert ocache.evict_aged(acc, np.arange(n), keep, first, recent, n).tolist() == ocache.evict(acc, keep, first, recent).tolist()


@pytest.mark.parametrize("keep,first,recent,over", [(2048, 4, 256, 64), (48, 2, 8, 1), (100, 0, 30, 40)])
def test_the_newest_stay_over_many_evictions(keep, first, recent, over):
    """Young tokens of little weight: all of the newest stay by age; by place those before the last call's are lost from
    the second eviction on."""
    left = {}
    for by_age in (True, False):
        rng = np.random.default_rng(1)
        born, acc, newest = np.arange(keep), np.exp(rng.standard_normal(keep)), keep
        for _ in range(14):
            born, newest = np.r_[born, np.arange(newest, newest + over)], newest + over
            acc = np.r_[acc, np.full(over, 1e-3)]
            src = ocache.evict_aged(acc, born, keep, first, recent, newest) if by_age else ocache.evict(acc, keep, first, recent)
            born, acc = born[src], acc[src]
            assert len(set(born.tolist())) == keep and born[:first].tolist() == list(range(first))
        left[by_age] = int((born >= newest - recent).sum())
    assert left[True] == recent and (left[False] < recent or over >= recent)


def test_workspace_over_another_array(lib):
    """The list of moves and the status word are written to the workspace while the arrays are in use."""
    p = _p()
    need = mita.mita_cache_evict_workspace_size(p)
    x = lambda a: None if a is None else ctypes.c_void_p(a)

    def plain(cache=2 * A, table=3 * A, lens=4 * A, keep=5 * A, acc=6 * A, len_out=7 * A, out=8 * A, src=9 * A):
        return lib.mita_cache_evict(p.ref, *map(x, (cache, table, lens, keep)), 0, 0, *map(x, (acc, len_out, out, src, 10 * A)),
                                    need, None)

    for name in ("cache", "table", "lens", "keep", "acc", "len_out", "out", "src"):
        for at in (10 * A, 10 * A + 1024, 10 * A + need - 16):
            assert plain(**{name: at}) == 1, (name, at)
            assert b"workspace" in lib.mita_last_error()
            assert _evict(lib, p, **{name: at}, n=need) == 1, (name, at)
    for at in (10 * A, 10 * A + need - 16):
        assert _evict(lib, p, age=at, n=need) == 1
    assert plain(acc=10 * A + 1024, out=10 * A + 1024) == 1  # in place


def test_table_that_is_the_lengths(lib):
    """len_out may be len, which a table of one column that starts there too does not become."""
    p = _p(max_pages=1)
    for kw in (dict(table=4 * A, lens=4 * A, len_out=4 * A), dict(keep=4 * A, lens=4 * A, len_out=4 * A)):
        assert _evict(lib, p, n=0, **kw) == 1, kw
    assert _evict(lib, p, n=0, lens=4 * A, len_out=4 * A) == 3


def test_numbers_beyond_32_bits(lib):
    """They would arrive as what their lower 32 bits say."""
    p = _p()
    cache, lens = torch.zeros(p.pool_bytes, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    table, acc, ws = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 2, 256), torch.zeros(4096, dtype=torch.uint8)
    for kw in (dict(first=2 ** 32), dict(recent=2 ** 32 + 5), dict(first=2 ** 31), dict(recent=-2 ** 31 - 1)):
        with pytest.raises(ValueError, match="first and recent"):
            mita.mita_cache_evict(p, cache, table, lens, lens.clone(), acc, ws, **kw)
    for args, kw in (((2 ** 32 + 64,), {}), ((64,), dict(scaling=2 ** 32, factor=2.0))):
        with pytest.raises(ValueError, match="32 bits"):
            mita.mita_rope_frequencies(*args, **kw)
