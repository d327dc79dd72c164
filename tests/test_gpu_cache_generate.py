"""The attention weight of cached tokens, and eviction by it, on the GPU against
the fp64 oracle (oracle/cache.py)."""
import math

import numpy as np
import pytest

from oracle import cache as ocache
from tests import parity
from tests.cache_cases import Pool

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


# -------------------------------------------------------------------- weights


def _weigh(pool, H, T, causal, counts=None, simt=False, scale=0.0, decay=1.0, seed=1, q=None, lse=None, acc="draw",
           in_place=False, check=True):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, d = len(pool.lens), pool.d
    p = mita.CacheParams(B, H, pool.Hkv, T, d, pool.page, pool.n_pages, pool.cols, scale,
                         (mita.FLAG_CAUSAL if causal else 0) | (mita.FLAG_SIMT if simt else 0), pool.p.dtype)
    g = torch.Generator().manual_seed(seed)
    Q = torch.randn((B, H, T, d), generator=g).to(pool.td).cuda() if q is None else q
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    ws = mita.cache_workspace(p)
    if lse is None:
        lse = torch.full((B, H, T), 7.0, dtype=torch.float32, device="cuda")
        mita.mita_cache_attention(p, Q, pool.cache, pool.table, pool.len_t, torch.empty_like(Q), ws, counts=cnt,
                                  exps=pool.exps, lse_out=lse)
    if isinstance(acc, str):
        acc = torch.rand((B, pool.Hkv, pool.cols * pool.page), generator=torch.Generator().manual_seed(seed + 99)).cuda()
        for b, n in enumerate(pool.lens):  # what own tokens' places and those behind the end hold is not read
            acc[b, :, max(0, n - (T if counts is None else counts[b])):] = float("nan")
    out = acc if in_place else torch.full((B, pool.Hkv, pool.cols * pool.page), 7.0, device="cuda")
    before = None if acc is None else acc.clone()
    ws.fill_(0xff)
    mita.mita_cache_weights(p, Q, pool.cache, pool.table, pool.len_t, lse, acc, ws, counts=cnt, exps=pool.exps,
                            decay=decay, acc_out=None if in_place else out)
    if check:
        mita.mita_device_status(ws)
    return Q, lse, before, out


def _check_weights(pool, H, T, causal, Q, lse, acc, out, counts=None, scale=0.0, decay=1.0, label=""):
    """|gpu - oracle| of a token's sum, counted from the roundings:
      - a score: (d + 4) 2^-23 of its size sum |q_c k_c| scale for the products' sum (which may cut) and the
        entries as halves, 2 2^-24 of it for the scale;
      - its difference to lse 2^-24, the factor log2(e) and its product 2^-23 of the difference, the
        exponential 2^-22: the weight's relative error, with differences up to 90;
      - the rows' additions and the old sum's product: 2^-23 of the sum each, in chains of at most the rows + 8."""
    sc, G, worst = scale or 1.0 / math.sqrt(pool.d), H // pool.Hkv, 0.0
    for b, n in enumerate(pool.lens):
        c = T if counts is None else counts[b]
        lim = [max(0, n - (c - 1 - t)) if causal else n for t in range(c)]
        K = pool.held(b, 0)
        for h in range(pool.Hkv):
            want, err = np.zeros(n), np.zeros(n)
            for head in range(h * G, (h + 1) * G):
                if c == 0:
                    break
                q, L = _np(Q[b, head, :c]), _np(lse[b, head, :c])
                w = ocache.weights(q, K[h], lim, L, sc)
                for t in range(c):
                    m = lim[t]
                    mag = sc * (np.abs(K[h][:m]) @ np.abs(q[t]))
                    z = (K[h][:m] @ q[t]) * sc
                    rel = (pool.d + 6) * 2.0 ** -23 * mag + 2.0 ** -22 * (np.minimum(np.abs(z - L[t]), 90) + 1) \
                        + 2.0 ** -24 * np.abs(L[t] if m else 0)
                    err[:m] += w[t, :m] * rel
                want += w.sum(0)
            if decay:
                old = max(0, n - c)
                want[:old] += np.float32(decay) * _np(acc[b, h, :old])
            err = err * 1.01 + (G * c + 8) * 2.0 ** -23 * want + 1e-37
            diff = np.abs(_np(out[b, h, :n]) - want)
            assert np.all(diff <= err), (label, b, h, float((diff / err).max()))
            worst = max(worst, float((diff / err).max()) if n else 0.0)
    parity.REPORT.append(("cache weights " + label, worst, 0.0, out.numel()))


def _behind(pool, out, before, in_place):
    """Places from the sequences' ends on are left as they were."""
    for b, n in enumerate(pool.lens):
        tail = out[b, :, n:]
        assert (tail.isnan().all() if in_place else (tail == 7.0).all())


CASES = [
    # dtype, d, page, H, Hkv, T, causal, lens, counts, exps, decay
    ("bf16", 128, 16, 1, 1, 1, False, [1], None, False, 1.0),
    ("bf16", 128, 64, 4, 4, 1, True, [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300], None, False, 0.5),
    ("bf16", 128, 64, 8, 2, 1, True, [5000, 0, 777], None, True, 1.0),
    ("bf16", 64, 48, 6, 2, 5, True, [40, 1000, 4, 129], [5, 3, 5, 0], False, 0.9),
    ("bf16", 128, 32, 16, 2, 3, True, [600, 2], [3, 2], True, 0.0),
    ("bf16", 64, 64, 10, 1, 8, True, [900, 3, 64], None, False, 1.0),   # rows without a key
    ("bf16", 128, 128, 3, 3, 40, True, [40, 200], None, False, 0.0),
    ("bf16", 64, 16, 5, 5, 2, False, [3000, 1, 257], [2, 2, 1], True, 1.0),
    ("bf16", 128, 64, 48, 1, 1, False, [5000, 0, 130, 128], None, False, 0.99),
    ("bf16", 128, 16, 64, 2, 3, True, [2500, 2, 100], [3, 3, 1], True, 1.0),
    ("bf16", 128, 32, 2, 2, 70, True, [300, 69, 71], [70, 70, 3], False, 1.0),
    ("bf16", 128, 48, 33, 1, 2, True, [1, 700], None, True, 0.0),
    ("bf16", 128, 16, 66, 1, 9, True, [600, 8, 9], [9, 9, 0], False, 1.0),   # 594 rows a head
    ("bf16", 64, 32, 32, 2, 17, False, [400, 129], [17, 5], True, 0.0),
    ("bf16", 128, 16, 6, 3, 1, True, [33, 5000, 0, 31], None, True, 0.9),    # two rows
    ("bf16", 64, 32, 2, 2, 2, True, [1, 2, 700, 65], [1, 2, 2, 0], False, 1.0),
    ("f32", 128, 48, 2, 1, 1, False, [900, 17], None, True, 1.0),
    ("f32", 64, 64, 3, 3, 2, True, [2, 3000, 129], [2, 1, 0], False, 0.5),
    ("bf16", 64, 64, 11, 1, 3, True, [1300, 30], None, False, 1.0),          # 33 rows: tiles of 128 tokens
    ("bf16", 128, 64, 64, 1, 4, True, [60000, 40], None, False, 1.0),        # several tiles of rows, for long
    ("bf16", 64, 32, 90, 1, 6, True, [9, 30001], [6, 5], False, 0.5),        # two passes over the rows
    ("f32", 128, 64, 50, 1, 6, False, [20000], None, False, 1.0),
    ("f32", 128, 64, 2, 2, 1, False, [1, 127, 700], None, True, 1.0),
    ("f32", 64, 16, 6, 2, 3, True, [500, 2, 33], [3, 3, 1], False, 0.75),
    ("f32", 128, 32, 8, 1, 1, True, [4000, 0], None, False, 1.0),
    ("f32", 128, 48, 24, 2, 11, True, [500, 140], [11, 2], True, 0.0),
    ("f32", 64, 16, 40, 1, 3, False, [260], None, False, 1.0),
]


@pytest.mark.parametrize("simt", [False, True], ids=["", "simt"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_d%d_p%d_H%d_%d_T%d" % c[:6])
def test_weights_match_oracle(case, simt):
    dtype, d, page, H, Hkv, T, causal, lens, counts, exps, decay = case
    ex = np.random.default_rng(2).integers(-3, 4, (2, Hkv)) if exps else None
    pool = Pool(lens, Hkv, d, page, dtype, seed=len(lens), exps=ex)
    for in_place in (False, True):
        Q, lse, acc, out = _weigh(pool, H, T, causal, counts, simt, decay=decay, in_place=in_place)
        _behind(pool, out, acc, in_place)
        _check_weights(pool, H, T, causal, Q, lse, acc, out, counts, decay=decay,
                       label="%s d%d H%d/%d T%d %s" % (dtype, d, H, Hkv, T, "simt" * simt))


@pytest.mark.parametrize("dtype,H,T,simt", [("bf16", 4, 1, False), ("bf16", 32, 3, False), ("f32", 8, 2, False),
                                            ("f32", 4, 2, True)])
def test_weights_sum_to_the_rows(dtype, H, T, simt):
    """Every row gives a weight of one in all, whatever its keys and the scale."""
    pool = Pool([333, 50, 1025], 2, 128, 64, dtype, seed=9)
    _, _, _, out = _weigh(pool, H, T, True, simt=simt, scale=0.4, decay=0.0, acc=None)
    for b, n in enumerate(pool.lens):
        s = _np(out[b, :, :n]).sum(1)
        # lse and the weights are each off by their scores' roundings: |z| up to 0.4 * 400 here, 140 2^-23 of it and 2^-21
        assert np.all(np.abs(s - H // 2 * T) <= H // 2 * T * 2 * (140 * 160 + 4) * 2.0 ** -23)


@pytest.mark.parametrize("dtype,H,d,T,simt", [("bf16", 4, 128, 3, False), ("bf16", 12, 64, 3, False), ("bf16", 64, 128, 3, False),
                                              ("f32", 4, 128, 3, False), ("f32", 40, 64, 3, False), ("f32", 4, 128, 3, True),
                                              ("bf16", 130, 128, 3, False), ("f32", 100, 128, 3, False)])
def test_unseen_and_bad_rows(dtype, H, d, T, simt):
    """NaN in keys reaches their own tokens' sums alone; rows with NaN or an infinity, or with a NaN
    for their lse, make NaN of the tokens that they see and of no others; a row that sees nothing is harmless."""
    import torch

    def make(rng, shape):
        K, V = Pool.rows(rng, shape)
        K[0, :, 60] = np.nan
        return K, V

    pool = Pool([62, 40, 2], 2, d, 16, dtype, make=make, seed=6)
    clean = Pool([62, 40, 2], 2, d, 16, dtype, seed=6, fill=0)
    Q, lse, _, want = _weigh(clean, H, T, True, simt=simt)
    _, _, _, out = _weigh(pool, H, T, True, simt=simt, lse=lse)
    assert out[0, :, 60].isnan().all()
    out[0, :, 60] = want[0, :, 60]
    assert torch.equal(out, want)
    # row 0 of sequence 2 sees nothing, whatever it holds
    bad, bad_lse = Q.clone(), lse.clone()
    bad[2, :, 0], bad_lse[2, :, 0] = float("nan"), float("nan")
    bad[1, 0, 1, 3] = float("inf")       # sees 39 tokens, head 0
    bad_lse[1, H - 1, 0] = float("nan")  # sees 38, head 1
    _, _, _, out = _weigh(clean, H, T, True, simt=simt, q=bad, lse=bad_lse)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    assert out[1, 0, :39].isnan().all() and torch.equal(out[1, 0, 39:], want[1, 0, 39:])
    assert out[1, 1, :38].isnan().all() and torch.equal(out[1, 1, 38:], want[1, 1, 38:])


@pytest.mark.parametrize("dtype,H", [("bf16", 4), ("bf16", 64), ("f32", 4), ("f32", 40)])
def test_large_scores_stay_weights(dtype, H):
    """Rows so large that lse cannot hold their scores' differences give weights of at most 1 each; tiny ones
    spread evenly."""
    import torch
    pool = Pool([333], 2, 128, 64, dtype, seed=9)
    mag = torch.tensor([1e-30, 1e30]).cuda().repeat(H // 2).view(1, H, 1, 1)
    Q = (torch.randn((1, H, 2, 128), generator=torch.Generator().manual_seed(2)).cuda() * mag).to(pool.td)
    _, _, _, out = _weigh(pool, H, 2, False, q=Q, decay=0.0, acc=None)
    o = _np(out[0, :, :333])
    even = H // 4 * 2 / 333.0
    assert np.all(o >= even * (1 - 64 * 2.0 ** -23)) and np.all(o <= even * (1 + 64 * 2.0 ** -23) + H // 4 * 2)


@pytest.mark.parametrize("B", [31, 32, 33, 128, 129, 700])
@pytest.mark.parametrize("H,T", [(2, 1), (10, 1), (36, 2)])
def test_batches_of_many_sequences(B, H, T):
    """Short sequences, most of them unlike, some without tokens, at the sizes where the search for a warp's place changes."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 90, B)]
    lens[0], lens[B // 2], lens[-1] = 0, 300, 0
    pool = Pool(lens, 2, 64, 16, "bf16", seed=4)
    Q, lse, acc, out = _weigh(pool, H, T, True, decay=0.5)
    _behind(pool, out, acc, False)
    _check_weights(pool, H, T, True, Q, lse, acc, out, decay=0.5, label="bf16 d64 B%d H%d T%d" % (B, H, T))


@pytest.mark.parametrize("dtype,H", [("bf16", 2), ("bf16", 8), ("bf16", 64), ("f32", 2), ("f32", 12), ("f32", 64)])
def test_rows_of_unlike_size(dtype, H):
    """Rows from a thousandth of the usual size to a thousand times it, side by side, some of zeros: each is as exact as
    among its like."""
    import torch
    pool = Pool([700, 129], 2, 128, 64, dtype, seed=12)
    gen = torch.Generator().manual_seed(3)
    Q = torch.randn((2, H, 2, 128), generator=gen) * 2.0 ** torch.randint(-10, 11, (2, H, 2, 1), generator=gen)
    Q[0, 0, 0] = 0
    Q[1, H - 1, 1, ::2] *= 2.0 ** -20
    Q = Q.to(pool.td).cuda()
    for scale in (0.0, 0.001):
        Q, lse, acc, out = _weigh(pool, H, 2, True, q=Q, scale=scale)
        _check_weights(pool, H, 2, True, Q, lse, acc, out, scale=scale, label="%s unlike rows H%d" % (dtype, H))


def test_weights_twice_and_any_split():
    """The same call gives the same bits, and a token's sum does not depend on the other sequences."""
    import torch
    for dtype, H, T in (("bf16", 8, 1), ("bf16", 4, 2), ("bf16", 40, 4), ("bf16", 256, 5), ("f32", 8, 3), ("f32", 40, 4)):
        pool = Pool([700, 33, 4000], 4, 128, 32, dtype, seed=5)
        Q, lse, acc, a = _weigh(pool, H, T, True)
        _, _, _, b = _weigh(pool, H, T, True)
        assert torch.equal(a, b)
        one = Pool([700], 4, 128, 32, dtype, seed=5)
        one.cache, one.table, one.n_pages, one.cols = pool.cache, pool.table[:1], pool.n_pages, pool.cols
        _, _, _, c = _weigh(one, H, T, True, q=Q[:1].contiguous(), lse=lse[:1].contiguous(), acc=acc[:1].contiguous())
        assert torch.equal(c[0, :, :700], a[0, :, :700])


@pytest.mark.parametrize("simt", [False, True], ids=["", "simt"])
@pytest.mark.parametrize("dtype,H,T", [("bf16", 2, 1), ("bf16", 6, 1), ("bf16", 40, 2), ("bf16", 160, 2), ("f32", 2, 1), ("f32", 6, 2),
                                       ("f32", 40, 2)])
def test_weights_out_of_range(dtype, H, T, simt):
    """Bad pages, lengths, counts and exponents are reported, and the other sequences' sums are right."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pool = Pool([300, 200, 129], 2, 128, 32, dtype, seed=8)
    Q, lse, acc, want = _weigh(pool, H, T, False, simt=simt)
    kw = dict(simt=simt, q=Q, lse=lse, acc=acc, check=False)
    p = mita.CacheParams(3, H, 2, T, 128, 32, pool.n_pages, pool.cols, flags=mita.FLAG_SIMT if simt else 0, dtype=pool.p.dtype)

    def run(table=None, lens=None, counts=None, exps=None):
        out, ws = torch.full_like(want, 7.0), mita.cache_workspace(p)
        mita.mita_cache_weights(p, Q, pool.cache, pool.table if table is None else table, pool.len_t if lens is None else lens,
                                lse, acc, ws, counts=counts, exps=exps, acc_out=out)
        with pytest.raises(mita.MitaError) as e:
            mita.mita_device_status(ws)
        assert e.value.status == 6
        mita.mita_device_status(ws)  # cleared
        return out

    table = pool.table.clone()
    for page in (-1, pool.n_pages, 2 ** 31 - 1):
        table[1, 2] = page
        out = run(table=table)
        assert torch.equal(out[[0, 2]], want[[0, 2]])
        assert (out[1, :, 64:96] == 7.0).all() and torch.equal(out[1, :, :64], want[1, :, :64])
    for n in (-1, pool.cols * 32 + 1):
        out = run(table=pool.table.clamp(max=0), lens=torch.tensor([300, n, 129], dtype=torch.int32).cuda())
    i = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    out = run(counts=i(T, T + 1, T))
    assert torch.equal(out[[0, 2]], want[[0, 2]])
    out = run(counts=i(T, -1, T))
    assert torch.equal(out[[0, 2]], want[[0, 2]])
    run(exps=i(0, 61, 0, 0).view(2, 2))


# ------------------------------------------------------------------- eviction


def _held_rows(pool, lens):
    """What the first lens[b] places of each sequence hold now: [B][2] arrays [H_kv, len, d]."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, T = len(lens), max(1, max(lens))
    p = mita.CacheParams(B, pool.Hkv, pool.Hkv, T, pool.d, pool.page, pool.n_pages, pool.cols, dtype=pool.p.dtype)
    ws = mita.cache_workspace(p)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    K, V = (torch.zeros((B, pool.Hkv, T, pool.d), dtype=pool.td, device="cuda") for _ in range(2))
    mita.mita_cache_read(p, pool.cache, pool.table, ln, K, V, ws, counts=ln, exps=pool.exps)
    mita.mita_device_status(ws)
    return K, V


def _sums(rng, shape, kind):
    a = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        a = rng.integers(0, 4, shape).astype(np.float32)
    elif kind == "equal":
        a[:] = 0.25
    elif kind == "special":
        pick = rng.random(shape)
        a[pick < 0.1], a[(pick >= 0.1) & (pick < 0.2)] = np.nan, -np.nan
        a[(pick >= 0.2) & (pick < 0.3)], a[(pick >= 0.3) & (pick < 0.4)] = np.inf, -np.inf
        a[(pick >= 0.4) & (pick < 0.5)], a[(pick >= 0.5) & (pick < 0.6)] = 0.0, -0.0
        a[(pick >= 0.6) & (pick < 0.7)] *= -1
        a[(pick >= 0.7) & (pick < 0.8)] = 1e-42  # below the normal numbers
    elif kind == "near":  # the last digits decide
        a = (1 + rng.integers(0, 64, shape) * 2.0 ** -23).astype(np.float32)
    return a


EVICT = [
    # d, page, Hkv, lens, keep, first, recent, sums, exps
    (128, 16, 1, [1], [1], 0, 0, "any", False),
    (128, 64, 2, [300, 64, 65, 0, 129], [64, 64, 64, 5, 128], 0, 0, "any", False),
    (64, 48, 3, [1000, 999, 31, 700], [100, 998, 31, 4], 4, 0, "any", True),
    (128, 32, 2, [500, 333], [150, 200], 10, 100, "any", False),
    (64, 16, 2, [500, 333, 10], [150, 200, 0], 0, 0, "ties", False),
    (128, 64, 1, [2000, 1500], [700, 1499], 1, 1, "equal", False),
    (64, 64, 2, [2000, 900], [700, 30], 0, 17, "special", False),
    (128, 16, 2, [3000], [1100], 16, 0, "near", True),
    (64, 16, 1, [400, 400], [60, 60], 20, 40, "any", False),   # nothing between stays
    (128, 128, 1, [70000, 3], [20001, 600], 4, 512, "any", False),
    (64, 64, 2, [40000, 33000], [39999, 1], 0, 1, "ties", False),
    (128, 16, 3, [5, 0, 17], [0, 0, 0], 0, 0, "any", False),
    (64, 128, 1, [400001, 50], [100000, 60], 3, 20, "ties", False),  # more than the blocks hold
    (64, 4096, 100, [30, 9000], [20, 4500], 2, 2, "any", False),     # many heads
]


@pytest.mark.parametrize("in_place", [False, True], ids=["", "in_place"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "d%d_p%d_H%d_n%d_%s" % (c[0], c[1], c[2], c[3][0], c[7]))
def test_eviction_matches_oracle(case, dtype, in_place):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    d, page, Hkv, lens, keep, first, recent, kind, exps = case
    rng = np.random.default_rng(len(lens) + d)
    ex = rng.integers(-9, 10, (2, Hkv)) if exps else None
    pool = Pool(lens, Hkv, d, page, dtype, seed=3, exps=ex)
    B, cap = len(lens), pool.cols * page
    sums = _sums(rng, (B, Hkv, cap), kind)
    acc = torch.from_numpy(sums).cuda()
    K0, V0 = _held_rows(pool, lens)
    keep_t = torch.tensor(keep, dtype=torch.int32).cuda()
    ws = mita.cache_evict_workspace(pool.p)
    ws.fill_(0xff)
    src = torch.full((B, Hkv, cap), -7, dtype=torch.int32, device="cuda")
    if in_place:
        n_out, a_out = pool.len_t.clone(), acc
        lens_in = n_out
    else:
        n_out, a_out = torch.full((B,), -7, dtype=torch.int32, device="cuda"), torch.full_like(acc, 7.0)
        lens_in = pool.len_t
    mita.mita_cache_evict(pool.p, pool.cache, pool.table, lens_in, keep_t, acc, ws, first=first, recent=recent,
                          len_out=None if in_place else n_out, acc_out=None if in_place else a_out, src_out=src)
    mita.mita_device_status(ws)
    now = [min(n, k) for n, k in zip(lens, keep)]
    assert n_out.tolist() == now
    K1, V1 = _held_rows(pool, lens)  # the whole sequences again: places from the new length on hold what they did
    bits = lambda t: t.cpu().numpy().view(np.int32)
    for b in range(B):
        for h in range(Hkv):
            want = ocache.evict(sums[b, h, :lens[b]], keep[b], first, recent)
            assert src[b, h, :now[b]].tolist() == want.tolist(), (b, h)
            assert (src[b, h, now[b]:] == -7).all()
            at = torch.from_numpy(np.concatenate([want, np.arange(now[b], lens[b])]).astype(np.int64)).cuda()
            for x, y in ((K0, K1), (V0, V1)):
                assert torch.equal(x[b, h][at].view(torch.int32 if dtype == "f32" else torch.int16),
                                   y[b, h, :lens[b]].view(torch.int32 if dtype == "f32" else torch.int16))
            np.testing.assert_array_equal(bits(a_out[b, h, :now[b]]), sums[b, h][want].view(np.int32))
            if in_place:
                np.testing.assert_array_equal(bits(a_out[b, h, now[b]:]), sums[b, h, now[b]:].view(np.int32))
            else:
                assert (a_out[b, h, now[b]:] == 7.0).all()


@pytest.mark.parametrize("kind", ["any", "near"])
def test_eviction_of_unaligned_sums(kind):
    """Sums that are aligned to their elements only."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    lens, keep = [5000, 33, 4997], [1234, 20, 4000]
    pool = Pool(lens, 2, 64, 16, "bf16", seed=3)
    cap = pool.cols * 16
    sums = _sums(np.random.default_rng(5), (3, 2, cap), kind)
    odd = lambda dt: torch.full((6 * cap + 1,), 7, dtype=dt, device="cuda")[1:].view(3, 2, cap)
    acc, out, src = odd(torch.float32), odd(torch.float32), odd(torch.int32)
    acc.copy_(torch.from_numpy(sums))
    ws = mita.cache_evict_workspace(pool.p)
    mita.mita_cache_evict(pool.p, pool.cache, pool.table, pool.len_t, torch.tensor(keep, dtype=torch.int32).cuda(), acc, ws,
                          recent=5, acc_out=out, src_out=src)
    mita.mita_device_status(ws)
    for b in range(3):
        for h in range(2):
            want = ocache.evict(sums[b, h, :lens[b]], keep[b], 0, 5)
            assert src[b, h, :keep[b]].tolist() == want.tolist()
            np.testing.assert_array_equal(out[b, h, :keep[b]].cpu().numpy(), sums[b, h][want])


def test_eviction_out_of_range():
    """A sequence with a bad length or budget is left as it is, one with a bad page moves its other rows; both are
    reported; the other sequences are cut as they should be."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    lens, rng = [300, 200, 129], np.random.default_rng(1)
    i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()

    def run(table=None, lens_=None, keep=(100, 100, 100), first=4, recent=8):
        pool = Pool(lens, 2, 64, 32, "bf16", seed=8)
        sums = _sums(rng, (3, 2, pool.cols * 32), "any")
        acc, src = torch.from_numpy(sums).cuda(), torch.full((3, 2, pool.cols * 32), -7, dtype=torch.int32, device="cuda")
        out, n_out = torch.full_like(acc, 7.0), i([-7] * 3)
        ws = mita.cache_evict_workspace(pool.p)
        t = pool.table.clone() if table is None else table(pool.table.clone(), pool)
        K0, V0 = _held_rows(pool, lens)
        mita.mita_cache_evict(pool.p, pool.cache, t, i(lens_ or lens), i(keep), acc, ws, first=first, recent=recent,
                              len_out=n_out, acc_out=out, src_out=src)
        with pytest.raises(mita.MitaError) as e:
            mita.mita_device_status(ws)
        assert e.value.status == 6
        K1, V1 = _held_rows(pool, lens)
        for b in (0, 2):
            for h in range(2):
                want = ocache.evict(sums[b, h, :lens[b]], keep[b], first, recent)
                assert src[b, h, :100].tolist() == want.tolist()
                at = torch.from_numpy(want.astype(np.int64)).cuda()
                assert torch.equal(K0[b, h][at], K1[b, h, :100]) and torch.equal(V0[b, h][at], V1[b, h, :100])
        return n_out.tolist(), src[1], out[1], (K0[1], V0[1]), (K1[1], V1[1])

    for bad in (-1, 1 << 20):
        n, src, out, before, after = run(lens_=[300, bad, 129])
        assert n == [100, bad, 100] and (src == -7).all() and (out == 7.0).all()
        assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    for bad in (11, -5):
        n, src, out, before, after = run(keep=(100, bad, 100))
        assert n == [100, 200, 100] and (src == -7).all() and (out == 7.0).all()
        assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])

    def page(col, value):
        def change(t, pool):
            t[1, col] = value if value is not None else pool.n_pages
            return t
        return change

    for col, value in ((1, -1), (5, None), (6, 2 ** 31 - 1)):
        n, src, out, before, after = run(table=page(col, value))
        assert n == [100] * 3
        moved = (src[:, :100] != torch.arange(100, device="cuda")).cpu().numpy()
        for h in range(2):
            for j in range(100):
                at = int(src[h, j])
                ok = j // 32 != col and at // 32 != col
                assert not ok or torch.equal(after[0][h, j], before[0][h, at])
                assert ok or not moved[h, j] or torch.equal(after[0][h, j], before[0][h, j])


def test_eviction_and_weights_captured():
    """A decoding loop in one graph: rotate, store, attend, weigh, evict; the lengths live on the device. Step by step the same
    as the calls one after the other."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, H, Hkv, d, page, budget = 3, 8, 2, 64, 16, 48
    start = [40, 46, 10]
    steps = 30
    gen = torch.Generator().manual_seed(7)
    rows = torch.randn((steps, B, 1, H + 2 * Hkv, d), generator=gen).to(torch.bfloat16).cuda()

    class Loop:
        def __init__(self):
            self.pool = Pool(start, Hkv, d, page, "bf16", seed=2, cols=6)
            pool = self.pool
            pool.n_pages = B * 6
            self.table = torch.arange(B * 6, dtype=torch.int32, device="cuda").view(B, 6)
            self.p = mita.CacheParams(B, H, Hkv, 1, d, page, B * 6, 6, flags=mita.FLAG_CAUSAL)
            self.fill = mita.CacheParams(B, Hkv, Hkv, max(start), d, page, B * 6, 6)
            self.cache = torch.zeros(mita.mita_cache_size(self.p), dtype=torch.uint8, device="cuda")
            self.lens = torch.tensor(start, dtype=torch.int32).cuda()
            mita.mita_cache_write(self.fill, pool.K, pool.V, self.cache, self.table, self.lens, mita.cache_workspace(self.fill),
                                  counts=self.lens)
            self.pos = self.lens.clone().view(B, 1)
            self.rope = mita.RopeParams(B, H, Hkv, 1, d, d)
            self.acc = torch.rand((B, Hkv, 96), generator=torch.Generator().manual_seed(1)).cuda()
            self.ws = [mita.cache_workspace(self.p) for _ in range(3)] + [mita.cache_evict_workspace(self.p)]
            for w in self.ws:
                w.fill_(0xff)
            self.x = torch.zeros((B, 1, H + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
            self.Q, self.O = (torch.zeros((B, H, 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.K, self.V = (torch.zeros((B, Hkv, 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.lse = torch.zeros((B, H, 1), device="cuda")
            self.keep = torch.full((B,), budget, dtype=torch.int32, device="cuda")

        def step(self):
            x = self.x.transpose(1, 2)
            mita.mita_rope(self.rope, x[:, :H], x[:, H:H + Hkv], self.Q, self.K, pos=self.pos)
            self.V.copy_(x[:, H + Hkv:])
            self.lens += 1
            self.pos += 1
            mita.mita_cache_write(self.p, self.K, self.V, self.cache, self.table, self.lens, self.ws[0])
            mita.mita_cache_attention(self.p, self.Q, self.cache, self.table, self.lens, self.O, self.ws[1], lse_out=self.lse)
            mita.mita_cache_weights(self.p, self.Q, self.cache, self.table, self.lens, self.lse, self.acc, self.ws[2], decay=0.9)
            mita.mita_cache_evict(self.p, self.cache, self.table, self.lens, self.keep, self.acc, self.ws[3], first=2, recent=8)

        def state(self):
            return [t.clone() for t in (self.cache, self.lens, self.acc, self.O, self.pos)]

    eager, captured = Loop(), Loop()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the modules load outside of the capture
        Loop().step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for t in range(steps):
        for loop in (eager, captured):
            loop.x.copy_(rows[t])
        eager.step()
        graph.replay()
        for w in eager.ws + captured.ws:
            mita.mita_device_status(w)
        for a, b in zip(eager.state(), captured.state()):
            assert torch.equal(a, b), t
        assert eager.lens.tolist() == [min(n + t + 1, budget) for n in start]


@pytest.mark.parametrize("H,T", [(2, 1), (12, 1), (48, 2), (200, 2)])
def test_weights_captured_and_beside_another_call(H, T):
    """A captured call reads its lengths when it is replayed; two calls on two streams at once, with a workspace each,
    give what they give one after the other."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pools = [Pool([5000, 300], 2, 128, 64, "bf16", seed=s) for s in (1, 2)]
    p = mita.CacheParams(2, H, 2, T, 128, 64, pools[0].n_pages, pools[0].cols, flags=mita.FLAG_CAUSAL)
    gen = torch.Generator().manual_seed(3)
    Q = torch.randn((2, H, T, 128), generator=gen).to(torch.bfloat16).cuda()
    lse = torch.full((2, H, T), 8.0, device="cuda")
    acc = torch.rand((2, 2, pools[0].cols * 64), generator=gen).cuda()
    wss = [mita.cache_workspace(p) for _ in pools]
    lens = [torch.tensor(x, dtype=torch.int32).cuda() for x in ([5000, 300], [4097, 1], [0, 129])]

    def call(i, ln, out, **kw):
        mita.mita_cache_weights(p, Q, pools[i].cache, pools[i].table, ln, lse, acc, wss[i], decay=0.5, acc_out=out, **kw)

    want = [[torch.zeros_like(acc) for _ in lens] for _ in pools]
    for i in range(2):
        for ln, out in zip(lens, want[i]):
            call(i, ln, out)
            mita.mita_device_status(wss[i])
    now, got = lens[0].clone(), torch.zeros_like(acc)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, now, got)
    for ln, w in zip(lens, want[0]):
        now.copy_(ln)
        got.zero_()
        graph.replay()
        mita.mita_device_status(wss[0])
        assert torch.equal(got, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(acc) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            call(i, lens[0], outs[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        mita.mita_device_status(wss[i])
        assert torch.equal(outs[i], want[i][0])


def test_eviction_beside_another_call():
    """Two evictions on two streams at once, with a workspace each, are as one after the other."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    res = []
    for at_once in (False, True):
        pools = [Pool([5000, 300], 2, 128, 64, "bf16", seed=s) for s in (1, 2)]
        accs = [torch.from_numpy(_sums(np.random.default_rng(s), (2, 2, p.cols * 64), "any")).cuda() for s, p in enumerate(pools)]
        keep = torch.tensor([777, 100], dtype=torch.int32).cuda()
        wss = [mita.cache_evict_workspace(p.p) for p in pools]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for p, a, w, s in zip(pools, accs, wss, streams):
            mita.mita_cache_evict(p.p, p.cache, p.table, p.len_t, keep, a, w, first=1, recent=2, stream=s)
            if not at_once:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        for w in wss:
            mita.mita_device_status(w)
        res.append([p.cache.clone() for p in pools] + accs + [p.len_t for p in pools])
    assert all(torch.equal(x, y) for x, y in zip(*res))
