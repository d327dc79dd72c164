"""Argument checks of rotation, cached tokens' weights and eviction, the
frequencies, and the oracles' own pins (no GPU: nothing here launches)."""
import copy
import ctypes
import pickle

import numpy as np
import pytest
import torch

import compressed_attention_adaptive_gb300 as mita
from compressed_attention_adaptive_gb300 import build as mita_build
from oracle import cache as ocache
from oracle import rope as orope

A = 1 << 20  # an address, never read


@pytest.fixture(scope="module")
def lib():
    mita_build.build()
    return mita.lib()


def _ptr(x):
    return None if x is None else ctypes.c_void_p(x)


# ------------------------------------------------------------------ rotation


def _r(**kw):
    base = dict(B=2, H=4, H_kv=2, T=3, d=64, rot=32)
    base.update(kw)
    return mita.RopeParams(**base)


def _rope(lib, p, Q=A, K=2 * A, Qo=3 * A, Ko=4 * A, strides=None, pos=None, ps=0, back=False):
    s = None if strides is None else (ctypes.c_int64 * 12)(*strides)
    fn = lib.mita_rope_backward if back else lib.mita_rope
    return fn(ctypes.byref(p) if isinstance(p, ctypes.Structure) else p.ref, _ptr(Q), _ptr(K), _ptr(Qo), _ptr(Ko), s,
              _ptr(pos), ps, None)


def _c(**kw):
    """The C parameters with plain frequencies, whatever kw makes of them."""
    c = mita._CRopeParams(B=2, H=4, H_kv=2, T=3, d=64, rot=32, dtype=mita.BF16)
    for i in range(mita.ROPE_PAIRS):
        c.freqs[i] = 1.0
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(H_kv=-1), 1), (dict(T=0), 1), (dict(d=0), 1), (dict(d=63), 1),
    (dict(d=258), 1), (dict(rot=0), 1), (dict(rot=31), 1), (dict(rot=66), 1), (dict(gain=float("nan")), 1),
    (dict(gain=float("inf")), 1), (dict(flags=1), 1), (dict(flags=4), 1), (dict(flags=16), 1), (dict(dtype=2), 1),
    (dict(H=65535), 2), (dict(B=1 << 20, T=1 << 20), 2),
])
def test_rope_parameters(lib, bad, status):
    for back in (False, True):
        assert _rope(lib, _c(**bad), back=back) == status
        assert lib.mita_last_error()


def test_rope_frequencies_must_be_finite(lib):
    for x in (float("nan"), float("inf")):
        c = _c()
        c.freqs[15] = x
        assert _rope(lib, c) == 1
        c.freqs[15], c.freqs[16] = 1.0, x  # past rot / 2: not read, so the next check speaks
        assert _rope(lib, c, Q=None) == 1 and b"device pointers" in lib.mita_last_error()
    assert lib.mita_rope(None, _ptr(A), _ptr(A), _ptr(A), _ptr(A), None, None, 0, None) == 1


def test_rope_pointers(lib):
    p = _r()
    for kw in (dict(Q=None), dict(K=None), dict(Qo=None), dict(Ko=None), dict(Q=A + 1), dict(Ko=4 * A + 1),
               dict(pos=5 * A + 2), dict(pos=5 * A, ps=-1)):
        assert _rope(lib, p, **kw) == 1, kw
    q = _r(H_kv=0)
    assert _rope(lib, q) == 1 and _rope(lib, q, Ko=None) == 1
    f = _r(dtype=mita.F32)
    assert _rope(lib, f, Q=A + 2) == 1


def _contiguous(H, T, d):
    return [H * T * d, T * d, d]


@pytest.mark.parametrize("what,kw", [
    ("outputs over each other", dict(Ko=3 * A + 2 * 100)),
    ("an output over the other input", dict(Qo=2 * A)),
    ("an output shifted over its own input", dict(Qo=A + 16)),
    ("in place with other strides", dict(Qo=A, strides=[768, 192, 64, 384, 192, 64, 768, 64, 256, 384, 192, 64])),
    ("negative stride", dict(strides=[768, 192, -64, 384, 192, 64, 768, 192, 64, 384, 192, 64])),
    ("rows of an output over each other", dict(strides=[768, 192, 64, 384, 192, 64, 768, 192, 32, 384, 192, 64])),
    ("an output that repeats a row", dict(strides=[768, 192, 64, 384, 192, 64, 0, 192, 64, 384, 192, 64])),
    ("an output over pos", dict(pos=3 * A + 8, ps=3)),
    ("keys inside the queries of a row", dict(Q=A, K=A + 2 * 128, Qo=A, Ko=A + 2 * 128,
                                              strides=[1536, 64, 512, 1536, 64, 512] * 2)),
])
def test_rope_overlaps_are_refused(lib, what, kw):
    for back in (False, True):
        assert _rope(lib, _r(), back=back, **kw) == 1, what
        assert lib.mita_last_error()


def test_rope_binding(lib):
    p = _r()
    q, k = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
    for args, kw in (((q, k, q, k), {}), ((q.float(), k, q, k), {}), ((q[:1], k, q, k), {}), ((q, k, q, k[:, :1]), {}),
                     ((q, None, q, k), {}), ((q.transpose(2, 3), k, q, k), {}),
                     ((q, k, q, k), dict(pos=torch.zeros(4, dtype=torch.int32))),
                     ((q, k, q, k), dict(pos=torch.zeros(2, 3, dtype=torch.int64)))):
        for fn in (mita.mita_rope, mita.mita_rope_backward):
            with pytest.raises(ValueError):
                fn(p, *args, **kw)
    with pytest.raises(ValueError):
        mita.RopeParams(1, 1, 1, 1, 64, 32, freqs=(1.0,)).ref
    with pytest.raises(mita.MitaError):
        mita.RopeParams(1, 1, 1, 1, 64, 33).ref
    p.ref
    assert copy.copy(p) == p and pickle.loads(pickle.dumps(p)) == p


@pytest.mark.parametrize("rot", [2, 10, 64, 128, 256])
@pytest.mark.parametrize("name,kw", [
    ("plain", {}), ("plain", dict(base=500000.0)), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
    ("parts", dict(factor=8.0, original=8192.0, low=1.0, high=4.0)),
    ("parts", dict(factor=32.0, original=100.0, low=0.0, high=0.5, base=1e6)),
])
def test_frequencies(lib, rot, name, kw):
    scaling = dict(plain=mita.ROPE_PLAIN, linear=mita.ROPE_LINEAR, ntk=mita.ROPE_NTK, parts=mita.ROPE_PARTS)[name]
    got = np.array(mita.mita_rope_frequencies(rot, scaling=scaling, **kw))
    want = orope.frequencies(rot, scaling=name, **kw).astype(np.float64)
    # double arithmetic: the exponent -2 i / rot and the base are each off by some 2^-53, which a logarithm of at
    # most ln(1e6 * 32^2) = 21 multiplies; pow itself, and the ramp, whose slope is at most original f / 2 pi / (high - low)
    np.testing.assert_allclose(got, want, rtol=64 * 2.0 ** -53 * (64 if name == "parts" else 1))
    assert got[0] == 1.0 or name == "linear" or (name == "parts" and rot > 0)


def test_frequency_refusals(lib):
    for kw in (dict(rot=0), dict(rot=3), dict(rot=258), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
               dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=2, factor=float("nan")),
               dict(scaling=3, factor=2.0, original=0.0), dict(scaling=3, factor=2.0, original=10.0, low=4.0, high=4.0),
               dict(scaling=2, factor=1e300)):
        with pytest.raises(mita.MitaError) as e:
            mita.mita_rope_frequencies(**{"rot": 64, **kw})
        assert e.value.status == 1
    assert lib.mita_rope_frequencies(None, 1e4, 0, 1.0, 0.0, 0.0, 1.0) == 1


def test_rope_oracle():
    """The oracle against complex numbers, its transpose and whole turns."""
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((3, 5, 20)), rng.integers(-1000, 1000, (3, 5))
    f = orope.frequencies(12)
    for il in (False, True):
        y = orope.rotate(x, pos, f, 12, il, gain=1.5)
        p, q = orope.pairs(12, il)
        z = (x[..., p] + 1j * x[..., q]) * 1.5 * np.exp(1j * pos[..., None] * f.astype(np.float64))
        np.testing.assert_allclose(y[..., p] + 1j * y[..., q], z, atol=1e-11)
        assert np.array_equal(y[..., 12:], x[..., 12:])
        g = rng.standard_normal(x.shape)
        np.testing.assert_allclose((orope.rotate(g, pos, f, 12, il, 1.5, back=True) * x).sum(), (g * y).sum(), rtol=1e-10)
    assert np.allclose(orope.rotate(x, 0, f, 12), x)


# -------------------------------------------------------- weights and eviction


def _p(**kw):
    base = dict(B=2, H=8, H_kv=2, T=1, d=128, page=64, n_pages=10, max_pages=4)
    base.update(kw)
    return mita.CacheParams(**base)


def _weigh(lib, p, Q=A, cache=2 * A, table=3 * A, lens=4 * A, counts=None, exps=None, lse=5 * A, decay=1.0, acc=6 * A,
           out=7 * A, ws=8 * A, n=1 << 40):
    return lib.mita_cache_weights(p.ref, *map(_ptr, (Q, cache, table, lens, counts, exps, lse)), decay, _ptr(acc),
                                  _ptr(out), _ptr(ws), n, None)


def _evict(lib, p, cache=2 * A, table=3 * A, lens=4 * A, keep=5 * A, first=0, recent=0, acc=6 * A, len_out=7 * A,
           out=8 * A, src=9 * A, ws=10 * A, n=1 << 40):
    return lib.mita_cache_evict(p.ref, *map(_ptr, (cache, table, lens, keep)), first, recent,
                                *map(_ptr, (acc, len_out, out, src, ws)), n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(H_kv=0), 1), (dict(T=0), 1), (dict(H=7), 1), (dict(d=100), 1), (dict(d=96), 2),
    (dict(page=8), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(dtype=5), 1), (dict(flags=1), 1),
    (dict(flags=8), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(B=65536), 2),
    (dict(n_pages=1 << 29), 2),
])
def test_cache_parameters(lib, bad, status):
    p = _p(**bad)
    assert _weigh(lib, p) == status and _evict(lib, p) == status
    assert mita.mita_cache_evict_workspace_size(p) == 0


def test_weights_pointers(lib):
    p = _p()
    need = mita.mita_cache_workspace_size(p)
    for kw in (dict(Q=None), dict(cache=None), dict(table=None), dict(lens=None), dict(lse=None), dict(out=None),
               dict(acc=None), dict(Q=A + 8), dict(cache=2 * A + 8), dict(table=3 * A + 2), dict(lens=4 * A + 1),
               dict(counts=A + 2), dict(exps=A + 2), dict(lse=5 * A + 2), dict(acc=6 * A + 1), dict(out=7 * A + 2),
               dict(decay=-1.0), dict(decay=float("nan")), dict(decay=float("inf")), dict(out=A), dict(out=5 * A),
               dict(out=6 * A + 4), dict(out=6 * A - 4), dict(out=2 * A + 64), dict(out=3 * A + 4), dict(out=4 * A),
               dict(out=9 * A, counts=9 * A + 4), dict(out=9 * A, exps=9 * A), dict(out=8 * A + 512)):
        assert _weigh(lib, p, **kw) == 1, kw
    for kw in (dict(ws=None), dict(ws=8 * A + 8), dict(n=need - 1)):
        assert _weigh(lib, p, **kw) == 3, kw
    assert _weigh(lib, p, acc=None, decay=0.0, n=need - 1) == 3  # acc may be absent then


def test_evict_pointers(lib):
    p = _p()
    need = mita.mita_cache_evict_workspace_size(p)
    assert need >= 1024 + 2 * 2 * 2 * 128 * 4
    for kw in (dict(cache=None), dict(table=None), dict(lens=None), dict(keep=None), dict(acc=None), dict(len_out=None),
               dict(out=None), dict(cache=2 * A + 8), dict(keep=5 * A + 2), dict(src=9 * A + 1), dict(first=-1),
               dict(recent=-1), dict(len_out=5 * A), dict(len_out=3 * A), dict(out=6 * A + 4), dict(src=6 * A),
               dict(src=8 * A), dict(len_out=8 * A), dict(src=2 * A), dict(out=4 * A), dict(len_out=4 * A + 4)):
        assert _evict(lib, p, **kw) == 1, kw
    for kw in (dict(ws=None), dict(ws=10 * A + 8), dict(n=need - 1), dict(src=None, n=0), dict(len_out=4 * A, n=0),
               dict(out=6 * A, n=0)):
        assert _evict(lib, p, **kw) == 3, kw


def test_cache_bindings(lib):
    p = _p()
    Q, cache = torch.zeros(2, 8, 1, 128, dtype=torch.bfloat16), torch.zeros(p.pool_bytes, dtype=torch.uint8)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    lse, acc, ws = torch.zeros(2, 8, 1), torch.zeros(2, 2, 256), torch.zeros(4096, dtype=torch.uint8)
    good = dict(Q=Q, cache=cache, table=table, lens=lens, lse=lse, acc=acc, ws=ws)
    for kw in ({}, dict(lse=lse[:1]), dict(acc=acc[..., :255]), dict(acc=acc.double()), dict(acc_out=acc[:1]),
               dict(Q=Q.float()), dict(cache=cache[:-1]), dict(acc=None)):
        with pytest.raises(ValueError):
            mita.mita_cache_weights(p, **{**good, **kw})
    good = dict(cache=cache, table=table, lens=lens, keep=lens.clone(), acc=acc, ws=ws)
    for kw in ({}, dict(keep=lens.long()), dict(acc=acc[:1]), dict(len_out=lens[:1]), dict(src_out=acc), dict(cache=cache[:-1]),
               dict(table=table[:1]), dict(acc_out=acc.half())):
        with pytest.raises(ValueError):
            mita.mita_cache_evict(p, **{**good, **kw})


def test_evict_oracle():
    acc = np.array([5.0, 1.0, 3.0, 3.0, 0.0, 9.0, 2.0, 3.0])
    # kept: 0 (first), 7 (recent), then 5 (9.0) and of the threes the lowest place, 2
    assert ocache.evict(acc, 4, 1, 1).tolist() == [0, 5, 2, 7]
    assert ocache.evict(acc, 8, 1, 1).tolist() == list(range(8))
    assert ocache.evict(acc, 20, 1, 1).tolist() == list(range(8))
    assert ocache.evict(acc, 2, 1, 1).tolist() == [0, 7]
    acc[4], acc[1] = np.nan, -0.0
    assert ocache.evict(acc, 2, 0, 0).tolist() == [4, 5] and ocache.evict(acc, 0, 0, 0).tolist() == []


def test_weights_oracle():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((3, 8)), rng.standard_normal((6, 8))
    _, lse, _ = ocache.attention(q, k, k, [6, 4, 0], 0.3)
    w = ocache.weights(q, k, [6, 4, 0], lse, 0.3)
    np.testing.assert_allclose(w.sum(1), [1, 1, 0], rtol=1e-12)
    assert (w[1, 4:] == 0).all() and (w[2] == 0).all()
