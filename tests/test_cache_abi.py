"""The cache calls' argument checks (no GPU: nothing here launches)."""
import copy
import ctypes
import pickle

import pytest
import torch

import compressed_attention_adaptive_gb300 as mita
from compressed_attention_adaptive_gb300 import build as mita_build


@pytest.fixture(scope="module")
def lib():
    mita_build.build()
    return mita.lib()


def _p(**kw):
    base = dict(B=2, H=8, H_kv=2, T=1, d=128, page=64, n_pages=10, max_pages=4)
    base.update(kw)
    return mita.CacheParams(**base)


def test_sizes(lib):
    assert mita.mita_cache_size(_p()) == 10 * 2 * 64 * (2 * (64 + 8))  # 9/16 byte per channel, keys and values
    assert mita.mita_cache_size(_p(d=64, page=16)) == 10 * 2 * 16 * (2 * (32 + 4))
    big = _p(n_pages=200000, H_kv=8)  # past 32 bits
    assert mita.mita_cache_size(big) == 200000 * 8 * 64 * 144
    assert mita.mita_cache_workspace_size(_p()) >= 1024


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(H_kv=0), 1), (dict(T=0), 1), (dict(H=7), 1), (dict(d=100), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(page=8), 1), (dict(page=40), 1), (dict(page=8192), 1),
    (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(dtype=5), 1), (dict(flags=1), 1), (dict(flags=8), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(B=65536), 2),
    (dict(T=1 << 29), 2), (dict(H=2 ** 31 - 2, H_kv=2), 2), (dict(max_pages=1 << 25), 2), (dict(n_pages=1 << 29), 2),
    (dict(B=1, H=1, H_kv=1, T=1 << 24, max_pages=1 << 14), 2),  # more work than 32 bits count
])
def test_invalid_parameters(lib, bad, status):
    p = _p(**bad)
    assert mita.mita_cache_size(p) == 0 and mita.mita_cache_workspace_size(p) == 0
    f, c = ctypes.c_void_p(1 << 20), ctypes.byref(p.c())
    big = 1 << 60
    assert lib.mita_cache_write(c, f, f, f, f, f, None, None, f, big, None) == status
    assert lib.mita_cache_read(c, f, f, f, None, None, f, f, f, big, None) == status
    assert lib.mita_cache_attention(c, f, f, f, f, None, None, f, None, f, big, None) == status
    assert lib.mita_last_error()


@pytest.mark.parametrize("kw", [
    dict(B=1, H=8, H_kv=8, T=1 << 20, d=64, n_pages=16384, max_pages=16384),
    dict(B=1, H=16, H_kv=16, T=1 << 20, n_pages=16384, max_pages=16384),
    dict(B=1, H=4, H_kv=4, T=1 << 20, n_pages=16384, max_pages=16384, dtype=mita.F32),
    dict(B=32, H=8, H_kv=8, T=131072, d=64, n_pages=65536, max_pages=2048, dtype=mita.F32),
])
def test_long_prompts_are_stored_whole(lib, kw):
    """The attention counts rows times tokens, storing and reading do not."""
    p = _p(**kw)
    c, f, odd = ctypes.byref(p.c()), ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
    assert mita.mita_cache_size(p) == p.pool_bytes
    need = mita.mita_cache_workspace_size(p)
    assert 0 < need <= 4096  # no partial results
    for n, k, status in ((need - 1, f, 3), (need, odd, 1)):  # past the parameters, to the checks behind them
        assert lib.mita_cache_write(c, k, f, f, f, f, None, None, f, n, None) == status
        assert lib.mita_cache_read(c, f, f, f, None, None, k, f, f, n, None) == status
    assert lib.mita_cache_attention(c, f, f, f, f, None, None, f, None, f, 1 << 60, None) == 2
    assert b"attention" in lib.mita_last_error()


def test_null_params(lib):
    f = ctypes.c_void_p(1 << 20)
    assert lib.mita_cache_size(None) == 0
    assert lib.mita_cache_write(None, f, f, f, f, f, None, None, f, 1 << 60, None) == 1


def test_pointers_and_workspace(lib):
    p = _p()
    c, need = ctypes.byref(p.c()), mita.mita_cache_workspace_size(p)
    f, odd, no = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8), ctypes.c_void_p((1 << 20) + 2)

    def write(K=f, V=f, cache=f, table=f, lens=f, counts=None, exps=None, ws=f, n=need):
        return lib.mita_cache_write(c, K, V, cache, table, lens, counts, exps, ws, n, None)

    def attend(Q=f, cache=f, table=f, lens=f, O=f, lse=None, ws=f, n=need):
        return lib.mita_cache_attention(c, Q, cache, table, lens, None, None, O, lse, ws, n, None)

    for kw in (dict(K=None), dict(V=None), dict(cache=None), dict(table=None), dict(lens=None), dict(K=odd),
               dict(cache=odd), dict(table=no), dict(lens=no), dict(counts=no), dict(exps=no)):
        assert write(**kw) == 1, kw
    for kw in (dict(Q=None), dict(O=None), dict(Q=odd), dict(O=odd), dict(lse=no)):
        assert attend(**kw) == 1, kw
    for fn in (write, attend):
        assert fn(ws=None) == 3
        assert fn(ws=odd) == 3
        assert fn(n=need - 1) == 3


def test_binding_checks_tensors(lib):
    """The C side sees pointers only, so the binding checks shapes, types and devices."""
    p = _p()
    K = torch.zeros((2, 2, 1, 128), dtype=torch.bfloat16)
    cache = torch.zeros(mita.mita_cache_size(p), dtype=torch.uint8)
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    ws = torch.zeros(mita.mita_cache_workspace_size(p), dtype=torch.uint8)
    ok = dict(K=K, V=K, cache=cache, table=table, lens=lens, ws=ws)
    for bad in (dict(K=K.float()), dict(V=K[:1]), dict(K=K.transpose(1, 2)[:, :, :1]), dict(table=table[:, :3]),
                dict(table=table.long()), dict(lens=lens[:1]), dict(counts=lens.long()), dict(exps=table),
                dict(cache=cache[:-1]), dict(cache=cache.view(torch.int8)), dict(ws=ws.view(torch.int8)),
                dict(table=table.t().contiguous().t())):
        with pytest.raises(ValueError):
            mita.mita_cache_write(p, **{**ok, **bad})
    with pytest.raises(ValueError, match="device"):  # host tensors of the right shapes
        mita.mita_cache_write(p, **ok)
    with pytest.raises(ValueError, match="device"):
        mita.mita_cache_read(p, cache, table, lens, K, K, ws)
    q = torch.zeros((2, 8, 1, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        mita.mita_cache_attention(p, q, cache, table, lens, q, ws)
    with pytest.raises(mita.MitaError):
        mita.cache_workspace(_p(d=96))


def test_overlapping_rows_are_refused(lib):
    """A part of O over Q would be read after it was written, and K over V written twice."""
    p = _p()
    c, need, at = ctypes.byref(p.c()), mita.mita_cache_workspace_size(p), 1 << 20
    f, q_bytes, k_bytes = ctypes.c_void_p(at), 2 * 8 * 128 * 2, 2 * 2 * 128 * 2
    for off in (0, 16, q_bytes - 16, -16, 16 - q_bytes):
        assert lib.mita_cache_attention(c, f, f, f, f, None, None, ctypes.c_void_p(at + off), None, f, need, None) == 1
        assert b"overlap" in lib.mita_last_error()
    for off in (0, k_bytes - 16, 16 - k_bytes):
        assert lib.mita_cache_read(c, f, f, f, None, None, f, ctypes.c_void_p(at + off), f, need, None) == 1
        assert b"overlap" in lib.mita_last_error()


def test_overlapping_log_sums_are_refused(lib):
    """A log sum over Q would be read as a query by blocks that come later, one over O be lost."""
    p = _p()
    c, need = ctypes.byref(p.c()), mita.mita_cache_workspace_size(p)
    Q, O, q_bytes, l_bytes = 1 << 20, (1 << 20) + (1 << 16), 2 * 8 * 128 * 2, 2 * 8 * 4
    f = ctypes.c_void_p(Q)
    for x in (Q, O):
        for lse in (x, x + q_bytes - 4, x + 4 - l_bytes):
            assert lib.mita_cache_attention(c, f, f, f, f, None, None, ctypes.c_void_p(O), ctypes.c_void_p(lse), f, need,
                                            None) == 1
            assert b"lse_out must not overlap" in lib.mita_last_error()


def test_params_copy_and_pickle_after_use(lib):
    p = _p(scale=0.25)
    mita.mita_cache_size(p)
    p.ref, p.pool_bytes
    for q in (copy.deepcopy(p), copy.copy(p), pickle.loads(pickle.dumps(p))):
        assert q == p and mita.mita_cache_size(q) == mita.mita_cache_size(p) == q.pool_bytes
