"""The 4-bit cache on the GPU against its fp64 oracle (oracle/cache.py).

What is stored is compared for equality (the format's two roundings are of exact
quotients); attention within bounds counted from its roundings
(tests/cache_cases.py), the oracle attending over the values it says the cache
holds.
"""
import math

import numpy as np
import pytest

from oracle import cache as ocache
from tests import parity
from tests.cache_cases import Pool, attention_bound

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------ write and read


@pytest.mark.parametrize("dtype,d,page,lens,counts,T,exps", [
    ("bf16", 128, 16, [1], None, 1, False),
    ("bf16", 128, 64, [5, 64, 65, 200], [5, 1, 2, 0], 7, True),
    ("bf16", 64, 48, [31, 95, 1, 17], [31, 40, 1, 16], 40, False),
    ("f32", 64, 16, [33, 16, 15], [33, 16, 0], 33, True),
    ("f32", 128, 4096, [700, 3], [1, 3], 3, False),
    ("bf16", 128, 112, [1000, 999], None, 999, True),
])
def test_rows_come_back_as_the_format_says(dtype, d, page, lens, counts, T, exps):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    Hkv = 3
    rng = np.random.default_rng(T)
    ex = rng.integers(-9, 10, (2, Hkv)).astype(np.int32) if exps else None
    # every row written, some by the fill and the last ones again with other values
    pool = Pool(lens, Hkv, d, page, dtype, seed=T, exps=ex, T=T)
    cnt = counts or [T] * len(lens)
    new = [rng.standard_normal((len(lens), Hkv, T, d)) * np.exp(rng.uniform(-3, 3, (len(lens), Hkv, T, 1)))
           for _ in range(2)]
    K, V = (torch.from_numpy(x).to(pool.td).cuda() for x in new)
    cnt_t = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    mita.mita_cache_write(pool.p, K, V, pool.cache, pool.table, pool.len_t, pool.ws, counts=cnt_t, exps=pool.exps)
    mita.mita_device_status(pool.ws)
    longest = max(lens)
    outs = [torch.full((len(lens), Hkv, longest, d), 7.0, dtype=pool.td, device="cuda") for _ in range(2)]
    mita.mita_cache_read(pool.fill_p, pool.cache, pool.table, pool.len_t, outs[0], outs[1], pool.fill_ws,
                         counts=pool.len_t, exps=pool.exps)
    mita.mita_device_status(pool.fill_ws)
    for which, (X, out) in enumerate(zip((K, V), outs)):
        for b, n in enumerate(lens):
            want = pool.held(b, which)
            c = cnt[b]
            if c:
                e = 0 if ex is None else ex[which][:, None]
                want[:, n - c:] = ocache.quantise(_np(X[b, :, :c]), e)
            np.testing.assert_array_equal(_np(out[b, :, :n]), want)
            assert torch.all(out[b, :, n:] == 7.0)  # padding rows left alone


def test_special_rows():
    import torch
    import compressed_attention_adaptive_gb300 as mita

    def make(rng, shape):
        x = rng.standard_normal(shape)
        x[0, 0, 0] = 0.0
        x[0, 0, 1] = -0.0
        x[0, 0, 2, 5] = np.nan
        x[0, 0, 3, 40] = np.inf
        x[0, 0, 4, 41] = -np.inf
        x[0, 0, 5] *= 1e30
        x[0, 0, 6] *= 1e-30
        x[0, 0, 7] *= 2.0 ** -12  # scales below e4m3's normal range
        x[0, 0, 8, :16] = np.r_[6.0, np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], 2), 6.0]  # ties, scale 1
        x[0, 0, 9, :16] = 2 * x[0, 0, 8, :16] * (-1.0) ** np.arange(16)
        x[0, 0, 10] = rng.integers(-40, 41, shape[-1])
        x[0, 0, 11, 2], x[0, 0, 11, 3] = np.nan, np.inf
        x[0, 0, 12] = 3.0e38
        return x, x[:, :, ::-1].copy()

    for dtype in ("bf16", "f32"):
        for ex in (None, [[0, 3], [-20, 1]]):
            pool = Pool([40], 2, 128, 16, dtype, make=make, exps=ex)
            K, V = (torch.empty_like(pool.K) for _ in range(2))
            mita.mita_cache_read(pool.fill_p, pool.cache, pool.table, pool.len_t, K, V, pool.fill_ws,
                                 counts=pool.len_t, exps=pool.exps)
            for which, out in enumerate((K, V)):
                np.testing.assert_array_equal(_np(out[0]), pool.held(0, which))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_next_to_midpoints(dtype, d):
    """Blocks whose largest channel is 6 times a midpoint between two scales, or one of
    the numbers next to it: the scale is that of the exact quotient, ties to even."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    big = (3 * (ocache.E4M3[1:] + ocache.E4M3[:-1])).astype(np.float32)
    step = 1 << 16 if dtype == "bf16" else 1
    big = (big.view(np.int32)[:, None] + step * np.arange(-2, 3, dtype=np.int32)).view(np.float32).ravel()
    n = -(-big.size // (d // 16))

    def make(rng, shape):
        x = rng.uniform(-1, 1, (n * (d // 16), 16)).astype(np.float32)
        x[:big.size] *= 0.99 * big[:, None]
        x[np.arange(big.size), rng.integers(0, 16, big.size)] = big * rng.choice(np.float32([-1, 1]), big.size)
        x = x.reshape(1, 1, n, d)
        return x, -x

    pool = Pool([n], 1, d, 16, dtype, make=make, seed=d)
    K, V = (torch.empty_like(pool.K) for _ in range(2))
    mita.mita_cache_read(pool.fill_p, pool.cache, pool.table, pool.len_t, K, V, pool.fill_ws)
    mita.mita_device_status(pool.fill_ws)
    for which, out in enumerate((K, V)):
        np.testing.assert_array_equal(_np(out[0]), pool.held(0, which))


def test_write_touches_only_its_places():
    """Storing a row changes that token's bytes and no others: every other token
    of the pool, of shared groups and of other pages too, reads as before."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pool = Pool([90, 70], 2, 64, 32, "bf16", T=1, seed=4)
    before = pool.cache.clone()
    K, V = (torch.randn((2, 2, 1, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    counts = torch.tensor([1, 0], dtype=torch.int32).cuda()
    mita.mita_cache_write(pool.p, K, V, pool.cache, pool.table, pool.len_t, pool.ws, counts=counts)
    mita.mita_device_status(pool.ws)
    changed = (pool.cache != before).view(-1)
    assert 0 < int(changed.sum()) <= 2 * 2 * (32 + 4)
    pages = torch.unique(changed.nonzero() // (changed.numel() // pool.n_pages))
    assert pages.tolist() == [int(pool.table[0, 89 // 32])]


# ---------------------------------------------------------------- attention


def _attend(pool, H, T, causal, counts=None, simt=False, scale=0.0, seed=1, lse=True, q=None):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, d = len(pool.lens), pool.d
    p = mita.CacheParams(B, H, pool.Hkv, T, d, pool.page, pool.n_pages, pool.cols, scale,
                         (mita.FLAG_CAUSAL if causal else 0) | (mita.FLAG_SIMT if simt else 0), pool.p.dtype)
    g = torch.Generator().manual_seed(seed)
    Q = torch.randn((B, H, T, d), generator=g).to(pool.td).cuda() if q is None else q
    O = torch.full_like(Q, 7.0)
    L = torch.full((B, H, T), 7.0, dtype=torch.float32, device="cuda") if lse else None
    ws = mita.cache_workspace(p)
    ws.fill_(0xff)
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    mita.mita_cache_attention(p, Q, pool.cache, pool.table, pool.len_t, O, ws, counts=cnt, exps=pool.exps, lse_out=L)
    mita.mita_device_status(ws)
    return Q, O, L


def _check(pool, H, T, causal, Q, O, L, counts=None, simt=False, scale=0.0, label=""):
    G, worst = H // pool.Hkv, 0.0
    sc = scale or 1.0 / math.sqrt(pool.d)
    for b, n in enumerate(pool.lens):
        c = T if counts is None else counts[b]
        assert (O[b, :, c:] == 7.0).all() and (L[b, :, c:] == 7.0).all()  # padding rows left alone
        if c == 0:
            continue
        K, V = pool.held(b, 0), pool.held(b, 1)
        lim = [max(0, n - (c - 1 - t)) if causal else n for t in range(c)]
        for h in range(H):
            k, v, q = K[h // G], V[h // G], _np(Q[b, h, :c])
            o, lse, spread = ocache.attention(q, k, v, lim, sc)
            bound = attention_bound(pool.dtype, pool.dtype == "bf16" and not simt, o, spread, q, k, v, lim, sc)
            diff = np.abs(_np(O[b, h, :c]) - o)
            assert np.all(diff <= bound), (label, b, h, float((diff / bound).max()))
            worst = max(worst, float((diff / bound).max()))
            got = L[b, h, :c].double().cpu().numpy()
            assert np.array_equal(got == -np.inf, lse == -np.inf)
            some = lse > -np.inf
            # the score's and the sum's relative errors become absolute ones
            mag = sc * np.abs(q) @ np.abs(k).max(0) if n else np.zeros(c)
            tol = (pool.d + 8) * 2.0 ** -23 * mag + (n / 16 + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -23 * np.abs(np.where(np.isinf(lse), 0, lse))
            assert np.all(np.abs(got[some] - lse[some]) <= tol[some])
    parity.REPORT.append(("cache attention " + label, worst, 0.0, O.numel()))


CASES = [
    # dtype, d, page, H, Hkv, T, causal, lens, counts, exps
    ("bf16", 128, 16, 1, 1, 1, False, [1], None, False),
    ("bf16", 128, 64, 4, 4, 1, True, [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300], None, False),
    ("bf16", 128, 64, 8, 2, 1, True, [5000, 0, 777], None, True),
    ("bf16", 64, 48, 6, 2, 5, True, [40, 1000, 4, 129], [5, 3, 5, 0], False),
    ("bf16", 128, 16, 16, 1, 1, False, [2049], None, False),
    ("bf16", 128, 32, 16, 2, 3, True, [600, 2], [3, 2], True),       # 24 rows a head: more than one tile
    ("bf16", 64, 64, 10, 1, 8, True, [900, 3, 64], None, False),     # 80 rows, rows without a key
    ("bf16", 128, 128, 3, 3, 40, True, [40, 200], None, False),      # a chunk of a prompt, rows in several tiles
    ("bf16", 64, 16, 5, 5, 2, False, [3000, 1, 257], [2, 2, 1], True),
    # more than 32 rows a head: tiles of 64
    ("bf16", 128, 64, 48, 1, 1, False, [5000, 0, 130, 128], None, False),
    ("bf16", 128, 16, 64, 2, 3, True, [2500, 2, 100], [3, 3, 1], True),
    ("bf16", 128, 32, 2, 2, 70, True, [300, 69, 71], [70, 70, 3], False),
    ("bf16", 128, 48, 33, 1, 2, True, [1, 700], None, True),
    ("f32", 128, 64, 2, 2, 1, False, [1, 127, 700], None, True),
    ("f32", 64, 16, 6, 2, 3, True, [500, 2, 33], [3, 3, 1], False),
    ("f32", 128, 32, 8, 1, 1, True, [4000, 0], None, False),
]


@pytest.mark.parametrize("simt", [False, True], ids=["", "simt"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_d%d_p%d_H%d_%d_T%d" % c[:6])
def test_attention_matches_oracle(case, simt):
    dtype, d, page, H, Hkv, T, causal, lens, counts, exps = case
    ex = np.random.default_rng(2).integers(-3, 4, (2, Hkv)) if exps else None
    pool = Pool(lens, Hkv, d, page, dtype, seed=len(lens), exps=ex)
    Q, O, L = _attend(pool, H, T, causal, counts, simt)
    _check(pool, H, T, causal, Q, O, L, counts, simt, label="%s d%d H%d/%d T%d %s" % (dtype, d, H, Hkv, T, "simt" * simt))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("lens,Hkv", [([380, 380], 3), ([1275], 1), ([1275, 500, 3], 2), ([5115], 1), ([5115, 0], 2),
                                      ([9000] * 2, 2)])
def test_few_and_many_parts(dtype, d, lens, Hkv):
    """Items that are cut into few parts, some and many: the join has a form for each."""
    pool = Pool(lens, Hkv, d, 48, dtype, seed=41)
    Q, O, L = _attend(pool, 3 * Hkv, 2, True)
    _check(pool, 3 * Hkv, 2, True, Q, O, L, label="parts %s d%d %s" % (dtype, d, lens))


@pytest.mark.parametrize("dtype,H", [("bf16", 4), ("bf16", 64), ("f32", 4)])
def test_scale_and_large_queries(dtype, H):
    """Scores far apart (one key takes all the weight), an explicit scale, and
    query rows of very unlike magnitude in one call."""
    import torch
    pool = Pool([333], 2, 128, 64, dtype, seed=9)
    mag = torch.tensor([1e-30, 1e-3, 1.0, 40.0]).cuda().repeat(H // 4).view(1, H, 1, 1)
    Q = torch.randn((1, H, 2, 128), generator=torch.Generator().manual_seed(2)).cuda() * mag
    Q[0, 1, 0] = 0
    Q = Q.to(pool.td)
    _, O, L = _attend(pool, H, 2, True, scale=0.5, q=Q)
    _check(pool, H, 2, True, Q, O, L, scale=0.5, label="scales %s H%d" % (dtype, H))


@pytest.mark.parametrize("dtype,H,d,simt", [("bf16", 4, 128, False), ("bf16", 12, 64, False), ("bf16", 64, 128, False),
                                            ("f32", 4, 128, False), ("f32", 4, 128, True)])
def test_unseen_keys_have_no_influence(dtype, H, d, simt):
    """A later drafted token full of NaN, and whatever bytes lie behind the last
    token: rows that do not see them are as without them, rows that do are NaN."""
    import torch
    T = 3

    def make(rng, shape):
        K, V = Pool.rows(rng, shape)
        K[0, :, 60], V[0, :, 60] = np.nan, np.nan     # the middle one of sequence 0's new tokens
        V[1, 0, 39, 16:32] = np.nan                   # one block of one head of sequence 1's last token
        K[2, 1, 5] = np.nan                           # a key that every row of sequence 2 sees
        return K, V

    pool = Pool([62, 40, 20], 2, d, 16, dtype, make=make, seed=6)
    Q, O, L = _attend(pool, H, T, True, simt=simt)
    clean = Pool([62, 40, 20], 2, d, 16, dtype, seed=6, fill=0)
    Q2, O2, L2 = _attend(clean, H, T, True, simt=simt)
    half = H // 2
    assert torch.equal(Q, Q2)
    assert torch.equal(O[0, :, 0], O2[0, :, 0]) and torch.equal(L[0, :, 0], L2[0, :, 0])
    assert O[0, :, 1:].isnan().all() and L[0, :, 1:].isnan().all()
    assert torch.equal(O[1, :, :2], O2[1, :, :2]) and torch.equal(O[1, half:, 2], O2[1, half:, 2])
    assert O[1, :half, 2, 16:32].isnan().all()
    assert torch.equal(O[1, :half, 2, :16], O2[1, :half, 2, :16])
    assert torch.equal(O[1, :half, 2, 32:], O2[1, :half, 2, 32:])
    assert O[2, half:].isnan().all() and torch.equal(O[2, :half], O2[2, :half])


@pytest.mark.parametrize("dtype,H,d", [("bf16", 8, 64), ("bf16", 40, 128), ("f32", 8, 128)])
def test_bad_rows_stay_in_their_rows(dtype, H, d):
    """NaN and infinite queries make their own rows NaN and no others."""
    import torch
    pool = Pool([150], 1, d, 16, dtype, seed=3)
    Q, O, L = _attend(pool, H, 2, False)
    bad = Q.clone()
    bad[0, 2, 1, 5], bad[0, 7, 0, 60] = float("nan"), float("inf")
    _, O2, _ = _attend(pool, H, 2, False, q=bad)
    hit = torch.zeros((H, 2), dtype=torch.bool)
    hit[2, 1] = hit[7, 0] = True
    assert O2[0][hit.cuda()].isnan().all()
    assert torch.equal(O2[0][~hit.cuda()], O[0][~hit.cuda()])


@pytest.mark.parametrize("dtype,H,d,simt", [("bf16", 8, 128, False), ("bf16", 24, 64, False), ("bf16", 64, 128, False),
                                            ("f32", 8, 128, False), ("f32", 16, 64, False), ("bf16", 8, 128, True)])
def test_rows_do_not_influence_each_other(dtype, H, d, simt):
    """Rows next to huge, tiny, infinite and NaN ones are the same bits as without them;
    a row with an infinity is NaN also where all of its scores are -infinity."""
    import torch

    def make(rng, shape):
        K, V = Pool.rows(rng, shape)
        K[..., 3] = 4 + np.abs(K[..., 3])
        return K, V

    pool = Pool([700, 33], 2, d, 16, dtype, make=make, seed=13)
    Q, O, L = _attend(pool, H, 2, True, simt=simt)
    bad = Q.clone()
    bad[:, 0::4, 0] *= 1e30
    bad[:, 1::4, 0] *= 1e-30
    bad[:, 2::4, 0, 3] = -math.inf
    bad[:, 3::4, 0, 3] = math.inf
    bad[:, 3::8, 0, 5] = math.nan
    _, O2, L2 = _attend(pool, H, 2, True, q=bad, simt=simt)
    assert torch.equal(O2[:, :, 1], O[:, :, 1]) and torch.equal(L2[:, :, 1], L[:, :, 1])
    for h in (2, 3):
        assert O2[:, h::4, 0].isnan().all() and L2[:, h::4, 0].isnan().all()
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    # the huge rows have the values of their largest score, up to scores that fp32 sums cannot tell from it
    for b, n in enumerate(pool.lens):
        for h in range(0, H, 4):
            k, v = (pool.held(b, w)[h // (H // 2), :n - 1] for w in (0, 1))
            q = _np(bad[b, h, 0])
            z, err = k @ q, (d + 8) * 2.0 ** -23 * (np.abs(k) @ np.abs(q)).max()
            top, got = v[z >= z.max() - 2 * err], _np(O2[b, h, 0])
            slack = (u + 100 * 2.0 ** -23) * np.abs(top).max(0)
            assert np.all(got >= top.min(0) - slack) and np.all(got <= top.max(0) + slack)
    # the tiny rows weigh all keys alike
    for b, n in enumerate(pool.lens):
        mean = np.stack([pool.held(b, 1)[h, :n - 1].mean(0) for h in range(2)]).repeat(H // 2, 0)
        spread = np.stack([np.abs(pool.held(b, 1)[h, :n - 1]).mean(0) for h in range(2)]).repeat(H // 2, 0)
        # the output's rounding; equal weights round alike; chains of fp32 additions and one quotient
        tol = u * np.abs(mean) + (n / 16 + 70) * 2.0 ** -23 * spread
        assert np.all(np.abs(_np(O2[b, :, 0]) - mean)[1::4] <= tol[1::4])


@pytest.mark.parametrize("dtype,H,d,simt", [("bf16", 4, 128, False), ("bf16", 24, 64, False), ("bf16", 64, 128, False),
                                            ("f32", 4, 128, False), ("f32", 24, 64, False), ("bf16", 4, 128, True),
                                            ("f32", 4, 64, True)])
def test_scores_near_the_lowest_float(dtype, H, d, simt):
    """Rows all of whose scores lie between the lowest float and half of it see their keys
    like any other: the keys with the largest score share the weight."""
    import torch

    def make(rng, shape):
        K, V = Pool.rows(rng, shape)
        K[..., :16] = 0
        K[..., 3] = rng.choice([4.0, 6.0], shape[:-1])
        K[0, 1, :, 3] = 6.0
        return K, V

    pool = Pool([700, 33, 1], 2, d, 16, dtype, make=make, seed=17)
    g = torch.Generator().manual_seed(4)
    Q = torch.randn((3, H, 2, d), generator=g).to(pool.td).cuda()
    _, O, L = _attend(pool, H, 2, True, simt=simt, scale=1.0, q=Q)
    low = Q.clone()
    low[:, 0::2, 1] = 0
    low[:, 0::2, 1, 3] = -3.7e37  # -2.1e38 and -3.2e38 in log2 units
    _, O2, L2 = _attend(pool, H, 2, True, simt=simt, scale=1.0, q=low)
    assert torch.equal(O2[:, 1::2], O[:, 1::2]) and torch.equal(O2[:, :, 0], O[:, :, 0])
    assert torch.equal(L2[:, 1::2], L[:, 1::2]) and torch.equal(L2[:, :, 0], L[:, :, 0])
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for b, n in enumerate(pool.lens):
        for h in range(0, H, 2):
            k, v = (pool.held(b, w)[h // (H // 2)] for w in (0, 1))
            z = k[:, 3] * float(low[b, h, 1, 3])
            best = z == z.max()
            mean, spread = v[best].mean(0), np.abs(v[best]).mean(0)
            # equal weights round alike; chains of fp32 additions and one quotient
            assert np.all(np.abs(_np(O2[b, h, 1]) - mean) <= u * np.abs(mean) + (n / 16 + 70) * 2.0 ** -23 * spread)
            # scale, log2(e) and ln(2) rounded, and the products
            assert abs(float(L2[b, h, 1]) / (z.max() + math.log(best.sum())) - 1) <= 8 * 2.0 ** -24


@pytest.mark.parametrize("simt", [False, True], ids=["", "simt"])
@pytest.mark.parametrize("d,T", [(64, 1), (128, 1), (64, 9), (128, 12)])
@pytest.mark.parametrize("gap", [24, 30, 36])
def test_float32_weights_far_below_the_largest(d, T, gap, simt):
    """A first key with 2^gap times the weight of the others and no values, as models have
    it: the result is what the others give, to float32."""

    def make(rng, shape):
        K, V = Pool.rows(rng, shape)
        K[..., :16] = 0
        K[:, :, 0, 0] = 6
        V[:, :, 0] = 0
        return K, V

    import torch
    pool = Pool([100, 4096, 700], 2, d, 64, "f32", make=make, seed=gap)
    Q = 0.1 * torch.randn((3, 2, T, d), generator=torch.Generator().manual_seed(gap))
    Q[..., 0] = gap * math.log(2) / 6
    Q = Q.cuda()
    _, O, L = _attend(pool, 2, T, False, simt=simt, scale=1.0, q=Q)
    for b, n in enumerate(pool.lens):
        for h in range(2):
            k, v, q = pool.held(b, 0)[h], pool.held(b, 1)[h], _np(Q[b, h])
            ref, lse, spread = ocache.attention(q, k, v, [n] * T, 1.0)
            # and 2^-48 of the largest weight where lower halves end
            bound = attention_bound("f32", False, ref, spread, q, k, v, [n] * T, 1.0) + 2.0 ** -48 * np.abs(v).sum(0)
            assert np.all(np.abs(_np(O[b, h]) - ref) <= bound), float((np.abs(_np(O[b, h]) - ref) / bound).max())


@pytest.mark.parametrize("H", [8, 64])
def test_repeated_calls_are_bit_equal_and_lse_is_optional(H):
    import torch
    pool = Pool([3000, 900], 2, 128, 64, "bf16", seed=12)
    runs = [_attend(pool, H, 2, True) for _ in range(3)]
    for _, O, L in runs[1:]:
        assert torch.equal(O, runs[0][1]) and torch.equal(L, runs[0][2])
    assert torch.equal(_attend(pool, H, 2, True, lse=False)[1], runs[0][1])


def test_pool_past_32_bits():
    """Pages more than 2^32 bytes into the pool."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    small = Pool([700, 90], 8, 128, 64, "bf16", seed=21, H=16)
    n_pages = 70000
    p = mita.CacheParams(2, 16, 8, 1, 128, 64, n_pages, small.cols)
    assert mita.mita_cache_size(p) > 2 ** 32 + 2 ** 29
    cache = torch.empty(mita.mita_cache_size(p), dtype=torch.uint8, device="cuda")
    table = torch.where(small.table < small.n_pages, n_pages - 1 - 3 * small.table, small.table)
    f = mita.CacheParams(2, 8, 8, 700, 128, 64, n_pages, small.cols)
    ws = mita.cache_workspace(f)
    mita.mita_cache_write(f, small.K, small.V, cache, table, small.len_t, ws, counts=small.len_t)
    mita.mita_device_status(ws)
    K, V = torch.zeros_like(small.K), torch.zeros_like(small.V)
    mita.mita_cache_read(f, cache, table, small.len_t, K, V, ws, counts=small.len_t)
    mita.mita_device_status(ws)
    for b, n in enumerate(small.lens):
        np.testing.assert_array_equal(_np(K[b, :, :n]), small.held(b, 0))
        np.testing.assert_array_equal(_np(V[b, :, :n]), small.held(b, 1))
    Q, O, L = _attend(small, 16, 1, False)
    for q in (p, mita.CacheParams(2, 16, 8, 1, 128, 64, n_pages, small.cols, flags=mita.FLAG_SIMT)):
        O2, w = torch.zeros_like(O), mita.cache_workspace(q)
        mita.mita_cache_attention(q, Q, cache, table, small.len_t, O2, w)
        mita.mita_device_status(w)
        if not q.flags:
            assert torch.equal(O, O2)
        else:
            assert torch.allclose(O.float(), O2.float(), rtol=2 ** -6, atol=2 ** -8)


def test_a_prompt_too_long_for_one_attention_call():
    """A million tokens stored and read back in one call each; attention takes as many
    tokens, but not as many rows at once."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    n, H, d, page = 1 << 20, 8, 64, 64
    p = mita.CacheParams(1, H, H, n, d, page, n // page, n // page)
    g = torch.Generator(device="cuda").manual_seed(3)
    K, V = (torch.randn((1, H, n, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cache = torch.zeros(mita.mita_cache_size(p), dtype=torch.uint8, device="cuda")
    table = torch.randperm(n // page, generator=g, device="cuda").to(torch.int32).view(1, -1)
    lens, ws = torch.tensor([n], dtype=torch.int32, device="cuda"), mita.cache_workspace(p)
    mita.mita_cache_write(p, K, V, cache, table, lens, ws)
    mita.mita_device_status(ws)
    outs = [torch.zeros_like(K) for _ in range(2)]
    mita.mita_cache_read(p, cache, table, lens, *outs, ws)
    mita.mita_device_status(ws)
    at = torch.cat([torch.arange(40), torch.randint(0, n, (2000,), generator=torch.Generator().manual_seed(1)),
                    torch.arange(n - 40, n)]).cuda()
    for X, out in zip((K, V), outs):
        np.testing.assert_array_equal(_np(out[0, :, at]), ocache.quantise(_np(X[0, :, at])))
    with pytest.raises(mita.MitaError) as err:
        mita.mita_cache_attention(p, K, cache, table, lens, torch.empty_like(K), ws)
    assert err.value.status == 2
    one = mita.CacheParams(1, H, H, 1, d, page, n // page, n // page)
    q, o = K[:, :, -1:].contiguous(), torch.zeros((1, H, 1, d), dtype=torch.bfloat16, device="cuda")
    w = mita.cache_workspace(one)
    mita.mita_cache_attention(one, q, cache, table, lens, o, w)
    mita.mita_device_status(w)
    for h in (0, H - 1):
        k, v, qq = _np(outs[0][0, h]), _np(outs[1][0, h]), _np(q[0, h])
        ref, _, spread = ocache.attention(qq, k, v, [n], 1 / math.sqrt(d))
        assert np.all(np.abs(_np(o[0, h]) - ref) <= attention_bound("bf16", True, ref, spread, qq, k, v, [n], 1 / math.sqrt(d)))


def test_tiles_past_32_bits():
    """The same for tiles of 64 rows, whose copies take several groups of a page."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    small = Pool([700, 90], 2, 128, 256, "bf16", seed=22, H=128)
    n_pages = 70000
    p = mita.CacheParams(2, 128, 2, 1, 128, 256, n_pages, small.cols)
    assert mita.mita_cache_size(p) > 2 ** 32 + 2 ** 29
    cache = torch.empty(mita.mita_cache_size(p), dtype=torch.uint8, device="cuda")
    table = torch.where(small.table < small.n_pages, n_pages - 1 - 3 * small.table, small.table)
    f = mita.CacheParams(2, 2, 2, 700, 128, 256, n_pages, small.cols)
    mita.mita_cache_write(f, small.K, small.V, cache, table, small.len_t, mita.cache_workspace(f), counts=small.len_t)
    Q, O, L = _attend(small, 128, 1, False)
    O2, ws = torch.zeros_like(O), mita.cache_workspace(p)
    mita.mita_cache_attention(p, Q, cache, table, small.len_t, O2, ws)
    mita.mita_device_status(ws)
    assert torch.equal(O, O2)


def test_many_short_sequences_and_shared_pages():
    """A thousand sequences, most of a few tokens, some without a row; then every
    second one with the pages of its neighbour (a shared prefix)."""
    import torch
    rng = np.random.default_rng(31)
    lens = [int(n) for n in np.where(rng.random(1000) < 0.9, rng.integers(0, 40, 1000), rng.integers(100, 900, 1000))]
    counts = [int(c) for c in rng.integers(0, 3, 1000)]
    pool = Pool(lens, 1, 64, 16, "bf16", seed=31)
    Q, O, L = _attend(pool, 2, 2, True, counts)
    _check(pool, 2, 2, True, Q, O, L, counts, label="1000 sequences")
    pool.table[1::2] = pool.table[0::2]
    pool.len_t[1::2] = pool.len_t[0::2]
    Q[1::2] = Q[0::2]
    _, O2, _ = _attend(pool, 2, 2, True, [c for c in counts[0::2] for _ in range(2)], q=Q)
    # equal sequences are cut at different places: two roundings to bf16 (2^-8 |o| each) and of
    # the weights to halves (2^-11 of at most max |v| < 4, each)
    a, b = O2[0::2].float(), O2[1::2].float()
    assert torch.all((a - b).abs() <= 2 * (2.0 ** -8 * a.abs().maximum(b.abs()) + 2.0 ** -11 * 4))


@pytest.mark.parametrize("dtype,d,H,T,B,simt", [("bf16", 128, 64, 1, 200, False), ("bf16", 128, 3, 5, 700, False),
                                                ("bf16", 64, 10, 2, 150, False), ("f32", 128, 1, 3, 300, False),
                                                ("f32", 64, 2, 1, 1400, False), ("bf16", 128, 2, 2, 150, True)])
def test_many_sequences_in_every_form(dtype, d, H, T, B, simt):
    """More sequences than a block's warps or threads, more items than pieces, empty ones among them."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 400 if B < 500 else 90, B) * rng.integers(0, 2, B)]
    lens[0], lens[-1] = 0, 700
    counts = [int(c) for c in rng.integers(0, T + 1, B)]
    counts[-1] = T
    pool = Pool(lens, 1, d, 16, dtype, seed=B)
    Q, O, L = _attend(pool, H, T, True, counts, simt)
    _check(pool, H, T, True, Q, O, L, counts, simt, label="%d sequences %s d%d%s" % (B, dtype, d, " simt" * simt))


@pytest.mark.parametrize("dtype,d,H,T", [("bf16", 128, 2, 1), ("bf16", 64, 6, 2), ("bf16", 128, 64, 2), ("f32", 64, 2, 3),
                                         ("f32", 128, 8, 4)])
def test_tensors_at_the_least_alignment(dtype, d, H, T):
    """Rows and pool 16 bytes past, index arrays and log sums 4 bytes past a larger boundary:
    the same bits, and nothing outside of the outputs is written."""
    import torch
    import compressed_attention_adaptive_gb300 as mita

    def shifted(t, by):
        n = t.numel() * t.element_size()
        buf = torch.full((n + 256,), 0x55, dtype=torch.uint8, device="cuda")
        x = buf[by:by + n].view(t.dtype).view(t.shape)
        x.copy_(t)
        assert x.data_ptr() % 256 == by
        return x, buf

    def kept(buf, x):
        n = x.numel() * x.element_size()
        at = x.data_ptr() - buf.data_ptr()
        return bool((buf[:at] == 0x55).all()) and bool((buf[at + n:] == 0x55).all())

    pool = Pool([300, 77], 2, d, 32, dtype, seed=2, exps=[[1, 2], [-1, 0]])
    Q, O, L = _attend(pool, H, T, True)
    K2, V2, Q2 = (shifted(x, 16)[0] for x in (pool.K, pool.V, Q))
    (cache, cb), (O2, ob), (L2, lb) = shifted(torch.zeros_like(pool.cache), 16), shifted(O, 16), shifted(L, 4)
    table, lens, exps = (shifted(x, 4)[0] for x in (pool.table, pool.len_t, pool.exps))
    O2.zero_(), L2.zero_()
    mita.mita_cache_write(pool.fill_p, K2, V2, cache, table, lens, pool.fill_ws, counts=lens, exps=exps)
    mita.mita_device_status(pool.fill_ws)
    outs = [shifted(torch.zeros_like(pool.K), 16) for _ in range(2)]
    mita.mita_cache_read(pool.fill_p, cache, table, lens, outs[0][0], outs[1][0], pool.fill_ws, counts=lens, exps=exps)
    mita.mita_device_status(pool.fill_ws)
    for which, (x, buf) in enumerate(outs):
        for b, n in enumerate(pool.lens):
            np.testing.assert_array_equal(_np(x[b, :, :n]), pool.held(b, which))
            assert (x[b, :, n:] == 0).all()
        assert kept(buf, x)
    p = mita.CacheParams(2, H, 2, T, d, 32, pool.n_pages, pool.cols, 0.0, mita.FLAG_CAUSAL, pool.p.dtype)
    ws = mita.cache_workspace(p)
    mita.mita_cache_attention(p, Q2, cache, table, lens, O2, ws, exps=exps, lse_out=L2)
    mita.mita_device_status(ws)
    assert torch.equal(O, O2) and torch.equal(L, L2)
    assert kept(cb, cache) and kept(ob, O2) and kept(lb, L2)


@pytest.mark.parametrize("dtype,d,H,simt", [("bf16", 128, 1, False), ("bf16", 128, 40, False), ("f32", 64, 1, False),
                                            ("bf16", 64, 1, True)])
def test_calls_without_rows(dtype, d, H, simt):
    """No sequence has a row, or a token: nothing is written, and the status word says so."""
    pool = Pool([50, 3, 0], 1, d, 16, dtype)
    Q, O, L = _attend(pool, H, 2, True, counts=[0, 0, 0], simt=simt)
    assert (O == 7).all() and (L == 7).all()
    empty = Pool([0, 0], 1, d, 16, dtype)
    for causal in (False, True):
        Q, O, L = _attend(empty, H, 2, causal, simt=simt)
        assert (O == 0).all() and (L == -math.inf).all()


@pytest.mark.parametrize("dtype,G,simt", [("bf16", 1, False), ("bf16", 40, False), ("f32", 2, False), ("bf16", 1, True)])
def test_as_many_sequences_as_a_call_takes(dtype, G, simt):
    """65535 sequences, most of a token or two: rows of some of them, and all of them
    against a call for the second half."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, d, page = 65535, 128 if G > 8 else 64, 16
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 4, B)
    lens[rng.integers(0, B, 300)] = rng.integers(1, 200, 300)
    lens[-1] = 130
    cols = -(-int(lens.max()) // page)
    need = -(-lens // page)
    table = np.full((B, cols), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in np.flatnonzero(need):
        table[b, :need[b]] = at[b] + np.arange(need[b])
    dt, td = (mita.F32, torch.float32) if dtype == "f32" else (mita.BF16, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(1)
    longest = int(lens.max())
    K, V = (torch.randn((B, 1, longest, d), generator=g, device="cuda").to(td) for _ in range(2))
    Q = torch.randn((B, G, 1, d), generator=g, device="cuda").to(td)
    table_t, len_t = torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda()
    f = mita.CacheParams(B, 1, 1, longest, d, page, int(at[-1]), cols, dtype=dt)
    cache, ws = torch.zeros(mita.mita_cache_size(f), dtype=torch.uint8, device="cuda"), mita.cache_workspace(f)
    mita.mita_cache_write(f, K, V, cache, table_t, len_t, ws, counts=len_t)
    mita.mita_device_status(ws)

    def attend(lo, hi):
        p = mita.CacheParams(hi - lo, G, 1, 1, d, page, int(at[-1]), cols, 0.0, mita.FLAG_SIMT * simt, dt)
        O, w = torch.full_like(Q[lo:hi], 7.0), mita.cache_workspace(p)
        mita.mita_cache_attention(p, Q[lo:hi].contiguous(), cache, table_t[lo:hi].contiguous(),
                                  len_t[lo:hi].contiguous(), O, w)
        mita.mita_device_status(w)
        return O

    O = attend(0, B)
    assert (O[torch.from_numpy(lens == 0).cuda()] == 0).all()
    # a sequence is cut at other places in the other call: the bound of _check, twice, with weights of at most 1
    half = attend(B // 2, B).float()
    tol = 2 * (2.0 ** -8 * half.abs() + 2.0 ** -11 * 6) if dtype == "bf16" else 2.0 ** -15
    assert torch.all((O[B // 2:].float() - half).abs() <= tol)
    for b in np.concatenate([[0, 1, B - 2, B - 1], rng.integers(0, B, 40), np.flatnonzero(lens > 100)[:20]]):
        n = int(lens[b])
        if n == 0:
            continue
        k, v = (ocache.quantise(_np(X[b, 0, :n])) for X in (K, V))
        q = _np(Q[b, :, 0])
        ref, _, spread = ocache.attention(q, k, v, [n] * G, 1 / math.sqrt(d))
        bound = attention_bound(dtype, dtype == "bf16" and not simt, ref, spread, q, k, v, [n] * G, 1 / math.sqrt(d))
        assert np.all(np.abs(_np(O[b, :, 0]) - ref) <= bound), b


# -------------------------------------------- out of range, and the status word


@pytest.mark.parametrize("what", ["page", "negative page", "len", "negative len", "count", "exps"])
def test_out_of_range_is_reported(what):
    """Each call reports it, leaves the other sequence right, and the next call
    on the same workspace is clean."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pool = Pool([100, 90], 2, 64, 32, "bf16", seed=8, T=2, H=4, exps=np.zeros((2, 2), int))
    ref = _attend(pool, 4, 2, True)
    table, lens = pool.table.clone(), pool.len_t.clone()
    counts, exps = torch.tensor([2, 2], dtype=torch.int32).cuda(), pool.exps.clone()
    if what == "page":
        table[0, 3] = pool.n_pages
    elif what == "negative page":
        table[0, 3] = -1
    elif what == "len":
        lens[0] = pool.cols * 32 + 1
    elif what == "negative len":
        lens[0] = -5
    elif what == "count":
        counts[0] = 3
    else:
        exps[0, 0] = 61
    K, V = (torch.randn((2, 2, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    cache = pool.cache.clone()
    O = torch.zeros_like(ref[1])
    p = mita.CacheParams(2, 4, 2, 2, 64, 32, pool.n_pages, pool.cols, 0.0, mita.FLAG_CAUSAL)
    calls = [lambda t, n, c, e: mita.mita_cache_write(p, K, V, cache, t, n, pool.ws, counts=c, exps=e),
             lambda t, n, c, e: mita.mita_cache_read(p, cache, t, n, K, V, pool.ws, counts=c, exps=e),
             lambda t, n, c, e: mita.mita_cache_attention(p, ref[0], pool.cache, t, n, O, pool.ws, counts=c, exps=e)]
    good = torch.tensor([2, 2], dtype=torch.int32).cuda()
    for call in calls:
        call(table, lens, counts, exps)
        with pytest.raises(mita.MitaError) as err:
            mita.mita_device_status(pool.ws)
        assert err.value.status == 6
    mine = slice(2, 4) if what == "exps" else slice(0, 4)  # an exponent belongs to a head, the rest to sequence 0
    assert torch.equal(O[1, mine], ref[1][1, mine])
    for call in calls:
        call(pool.table, pool.len_t, good, pool.exps)
        mita.mita_device_status(pool.ws)
    assert torch.equal(O, ref[1])


FORMS = [("bf16", 128, 1, 1), ("bf16", 64, 1, 5), ("bf16", 128, 6, 2), ("bf16", 64, 3, 10), ("bf16", 128, 32, 2),
         ("bf16", 128, 5, 40), ("f32", 128, 1, 1), ("f32", 64, 6, 3)]  # dtype, d, query heads a cache head, T


@pytest.mark.parametrize("simt", [False, True], ids=["", "simt"])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "%s_d%d_G%d_T%d" % f)
def test_out_of_range_in_every_form(form, simt):
    """Each form of the attention reports each kind of number that is out of range, leaves
    the sequences and heads that have none right, and is clean afterwards."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    dtype, d, G, T = form
    lens, Hkv, page = [700, 333, 450], 2, 48
    H = G * Hkv
    pool = Pool(lens, Hkv, d, page, dtype, seed=9, T=T, H=H, exps=np.array([[1, -2], [0, 3]]))
    flags = mita.FLAG_CAUSAL | (mita.FLAG_SIMT if simt else 0)
    p = mita.CacheParams(3, H, Hkv, T, d, page, pool.n_pages, pool.cols, 0.0, flags, pool.p.dtype)
    Q, O, L = _attend(pool, H, T, True, simt=simt)
    _check(pool, H, T, True, Q, O, L, simt=simt, label="in range, %s d%d G%d T%d" % form)
    counts = torch.full((3,), T, dtype=torch.int32, device="cuda")
    ws = mita.cache_workspace(p)
    sc = 1.0 / math.sqrt(d)

    def call(table=pool.table, lens=pool.len_t, counts=counts, exps=pool.exps):
        out, lse = torch.full_like(O, 7.0), torch.full_like(L, 7.0)
        mita.mita_cache_attention(p, Q, pool.cache, table, lens, out, ws, counts=counts, exps=exps, lse_out=lse)
        return out, lse

    def with_(t, at, v):
        t = t.clone()
        t[at] = v
        return t

    def bounds(b, h):
        n, lim = lens[b], [max(0, lens[b] - (T - 1 - t)) for t in range(T)]
        k, v, q = pool.held(b, 0)[h // G], pool.held(b, 1)[h // G], _np(Q[b, h])
        ref, _, spread = ocache.attention(q, k, v, lim, sc)
        off = attention_bound(dtype, dtype == "bf16" and not simt, ref, spread, q, k, v, lim, sc)
        return ref - off, ref + off

    # the first and the last query head of each cache head
    right = {(b, h): bounds(b, h) for b in range(3) for h in {0, G - 1, G, H - 1}}
    # the entry of a page in the middle, of the first and of the last one of sequence 1
    bad = [("page", dict(table=with_(pool.table, (1, i), v))) for i, v in ((3, pool.n_pages), (0, -1), (6, 2 ** 31 - 1))]
    bad += [("len", dict(lens=with_(pool.len_t, 1, v))) for v in (pool.cols * page + 1, -1, 2 ** 31 - 1)]
    bad += [("count", dict(counts=with_(counts, 1, v))) for v in (T + 1, -3)]
    bad += [("exps", dict(exps=with_(pool.exps, (w, 1), v))) for w, v in ((0, 61), (1, -61))]
    for what, kw in bad:
        out, _ = call(**kw)
        with pytest.raises(mita.MitaError) as err:
            mita.mita_device_status(ws)
        assert err.value.status == 6, what
        for (b, h), (lo, hi) in right.items():
            if h < G if what == "exps" else b != 1:  # an exponent belongs to a cache head, the rest to sequence 1
                got = _np(out[b, h])
                assert np.all((lo <= got) & (got <= hi)), (what, b, h)
    out, lse = call()
    mita.mita_device_status(ws)
    assert torch.equal(out, O) and torch.equal(lse, L)


def test_more_rows_than_tokens():
    """count > len: an error for the calls that store and read rows, rows without
    keys for attention."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pool = Pool([2, 5], 1, 64, 16, "bf16", T=4)
    K = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    before = pool.cache.view(pool.n_pages, -1).clone()
    mita.mita_cache_write(pool.p, K, K, pool.cache, pool.table, pool.len_t, pool.ws,
                          counts=torch.tensor([3, 0], dtype=torch.int32).cuda())
    with pytest.raises(mita.MitaError):
        mita.mita_device_status(pool.ws)
    changed = (pool.cache.view(pool.n_pages, -1) != before).any(dim=1).nonzero().view(-1).tolist()
    assert changed == [int(pool.table[0, 0])]  # the rows that have a place
    pool = Pool([2, 5], 1, 64, 16, "bf16", T=4)
    Q, O, L = _attend(pool, 1, 4, True)
    _check(pool, 1, 4, True, Q, O, L, label="more rows than tokens")
    assert torch.all(O[0, 0, :2] == 0) and torch.all(L[0, 0, :2] == -math.inf)


def test_the_status_word_is_the_last_calls():
    """A write's verdict is there until another call on its workspace: a workspace for each
    call keeps it, one for both has the attention's."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pool = Pool([2, 5], 1, 64, 16, "bf16", T=4)
    K = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    O, other = torch.zeros_like(K), mita.cache_workspace(pool.p)

    def step(ws):  # stores four rows of a sequence of two, which the attention may have
        mita.mita_cache_write(pool.p, K, K, pool.cache, pool.table, pool.len_t, pool.ws)
        mita.mita_cache_attention(pool.p, K, pool.cache, pool.table, pool.len_t, O, ws)

    step(other)
    mita.mita_device_status(other)
    with pytest.raises(mita.MitaError) as err:
        mita.mita_device_status(pool.ws)
    assert err.value.status == 6
    step(pool.ws)
    mita.mita_device_status(pool.ws)


@pytest.mark.parametrize("dtype,H,simt", [("bf16", 1, False), ("bf16", 12, False), ("f32", 1, False), ("bf16", 1, True)])
def test_more_rows_than_tokens_that_see_all(dtype, H, simt):
    """Without the causal flag rows have no position: each sees all keys, however many rows there are."""
    pool = Pool([2, 5, 0], 1, 128, 16, dtype)
    Q, O, L = _attend(pool, H, 4, False, simt=simt)
    _check(pool, H, 4, False, Q, O, L, simt=simt, label="more rows than tokens, all seen")
    assert (O[0] != 0).any(-1).all() and L[0].isfinite().all()
    assert (O[2] == 0).all() and (L[2] == -math.inf).all()


def test_binding_refuses():
    """Shapes, types and devices that the pointers of the C side cannot show."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pool = Pool([20, 5], 2, 64, 16, "bf16", H=4)
    Q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    ok = dict(Q=Q, cache=pool.cache, table=pool.table, lens=pool.len_t, O=torch.zeros_like(Q), ws=pool.ws)
    for bad in (dict(Q=Q.float()), dict(O=Q[:, :2]), dict(Q=Q.cpu()), dict(lens=pool.len_t.cpu()),
                dict(table=pool.table.long()), dict(cache=pool.cache[:-1]), dict(ws=pool.ws.cpu()),
                dict(counts=pool.len_t[:1]), dict(exps=pool.table[:1]), dict(lse_out=torch.zeros(2, 4, 1)),
                dict(lse_out=torch.zeros((2, 4, 1), dtype=torch.float64, device="cuda")),
                dict(lse_out=torch.zeros((2, 1, 4), device="cuda"))):
        with pytest.raises(ValueError):
            mita.mita_cache_attention(pool.p, **{**ok, **bad})
    with pytest.raises(mita.MitaError) as err:
        mita.mita_cache_attention(pool.p, **{**ok, "ws": pool.ws[:512]})
    assert err.value.status == 3
    mita.mita_cache_attention(pool.p, **ok)
    mita.mita_device_status(pool.ws)


# ------------------------------------------------------- streams and graphs


def test_captured_calls_follow_lengths_and_tables():
    """A captured step (write, then attend) replayed with other lengths, pages and
    rows; two captured graphs with their own workspaces replayed at once."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pools = [Pool([224, 224], 2, 128, 32, "bf16", seed=s, T=1, H=4) for s in (1, 2)]
    steps = []
    for pool in pools:
        st = dict(pool=pool, Q=torch.randn((2, 4, 1, 128)).cuda().to(torch.bfloat16),
                  K=torch.randn((2, 2, 1, 128)).cuda().to(torch.bfloat16),
                  V=torch.randn((2, 2, 1, 128)).cuda().to(torch.bfloat16))
        st["O"] = torch.zeros_like(st["Q"])

        def step(st=st, pool=pool):
            mita.mita_cache_write(pool.p, st["K"], st["V"], pool.cache, pool.table, pool.len_t, pool.ws)
            mita.mita_cache_attention(pool.p, st["Q"], pool.cache, pool.table, pool.len_t, st["O"], pool.ws)

        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        steps.append((st, step, graph, side))
    torch.cuda.synchronize()
    for lens in ([61, 201], [64, 17], [1, 224]):
        for st, step, graph, side in steps:
            st["pool"].len_t.copy_(torch.tensor(lens, dtype=torch.int32))
            for x in ("Q", "K", "V"):
                st[x].normal_()
            st["pool"].table.copy_(st["pool"].table.flip(0))
        torch.cuda.synchronize()
        for st, step, graph, side in steps:
            with torch.cuda.stream(side):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for st, step, graph, side in steps:
            got = st["O"].clone()
            mita.mita_device_status(st["pool"].ws)
            step()
            mita.mita_device_status(st["pool"].ws)
            assert got.isfinite().all() and torch.equal(got, st["O"])


def test_another_stream():
    import torch
    import compressed_attention_adaptive_gb300 as mita
    pool = Pool([500], 2, 64, 64, "bf16", H=2)
    Q = torch.randn((1, 2, 1, 64)).cuda().to(torch.bfloat16)
    a, b = torch.zeros_like(Q), torch.zeros_like(Q)
    mita.mita_cache_attention(pool.p, Q, pool.cache, pool.table, pool.len_t, a, pool.ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mita.mita_cache_attention(pool.p, Q, pool.cache, pool.table, pool.len_t, b, pool.ws, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


# --------------------------------------------------------- a run of them together


def test_beside_a_forward_pass_on_another_stream():
    """Attention of each form beside mita_forward on another stream is the same bits as alone."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    g = torch.Generator(device="cuda").manual_seed(5)
    X = [torch.randn((1, 4, 8192, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    fp = mita.Params(1, 4, 8192, 128, m=128, k=256, s=2)
    fws, FO = mita.workspace(fp), torch.empty_like(X[0])
    mita.mita_forward(fp, *X, FO, fws)
    want = FO.clone()
    calls = []
    for H, T, lens in ((2, 1, [3000, 500]), (16, 8, [2000, 900]), (128, 1, [4000, 700])):
        pool = Pool(lens, 2, 128, 64, "bf16", seed=H)
        Q, O, _ = _attend(pool, H, T, True)
        p = mita.CacheParams(2, H, 2, T, 128, 64, pool.n_pages, pool.cols, 0.0, mita.FLAG_CAUSAL)
        calls.append((pool, p, Q, O, torch.zeros_like(O), mita.cache_workspace(p)))
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        mita.mita_forward(fp, *X, FO, fws, stream=one)
        for pool, p, Q, O, O2, ws in calls:
            mita.mita_cache_attention(p, Q, pool.cache, pool.table, pool.len_t, O2, ws, stream=two)
    torch.cuda.synchronize()
    mita.mita_device_status(fws)
    # (its buckets fill in any order, so it is held to its own tolerance)
    assert torch.allclose(FO.float(), want.float(), rtol=2e-2, atol=2e-2)
    for _, _, _, O, O2, ws in calls:
        mita.mita_device_status(ws)
        assert torch.equal(O, O2)


def test_prompt_then_steps_then_another_pass():
    """A prompt through mita_forward, its keys and values stored, steps of one and
    of two tokens that store and attend, and at the end the whole sequences read
    back for another forward pass."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, H, Hkv, d, N, page, steps = 2, 4, 4, 128, 512, 64, [1, 1, 2, 1]
    total = N + sum(steps)
    g = torch.Generator().manual_seed(5)
    allK, allV, allQ = (torch.randn((B, H, total, d), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    cols = -(-total // page)
    table = torch.randperm(B * cols, generator=g).to(torch.int32).view(B, cols).cuda()
    mk = lambda T: mita.CacheParams(B, H, Hkv, T, d, page, B * cols, cols, flags=mita.FLAG_CAUSAL)
    cache = torch.zeros(mita.mita_cache_size(mk(1)), dtype=torch.uint8, device="cuda")
    ws = mita.cache_workspace(mk(N))
    part = lambda x, lo, hi: x[:, :, lo:hi].contiguous()
    O = mita.forward(part(allQ, 0, N), part(allK, 0, N), part(allV, 0, N), 16, 64, 2)
    assert O.isfinite().all()
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    mita.mita_cache_write(mk(N), part(allK, 0, N), part(allV, 0, N), cache, table, lens, ws)
    mita.mita_device_status(ws)
    heldK, heldV = (ocache.quantise(_np(x)) for x in (allK, allV))
    at = N
    for T in steps:
        p = mk(T)
        lens += T
        q, o = part(allQ, at, at + T), torch.zeros((B, H, T, d), dtype=torch.bfloat16, device="cuda")
        w = mita.cache_workspace(p)
        mita.mita_cache_write(p, part(allK, at, at + T), part(allV, at, at + T), cache, table, lens, w)
        mita.mita_cache_attention(p, q, cache, table, lens, o, w)
        mita.mita_device_status(w)
        at += T
        lim = [at - (T - 1 - t) for t in range(T)]
        for b in range(B):
            for h in range(H):
                k, v, qq = heldK[b, h, :at], heldV[b, h, :at], _np(q[b, h])
                ref, _, spread = ocache.attention(qq, k, v, lim, 1 / math.sqrt(d))
                bound = attention_bound("bf16", True, ref, spread, qq, k, v, lim, 1 / math.sqrt(d))
                assert np.all(np.abs(_np(o[b, h]) - ref) <= bound)
    full = mk(total)
    K, V = (torch.zeros((B, H, total, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = mita.cache_workspace(full)
    mita.mita_cache_read(full, cache, table, lens, K, V, w)
    mita.mita_device_status(w)
    np.testing.assert_array_equal(_np(K), heldK)
    np.testing.assert_array_equal(_np(V), heldV)
    again = mita.forward(allQ, K, V, 16, 64, 2)
    want = mita.forward(allQ, torch.from_numpy(heldK).to(torch.bfloat16).cuda(),
                        torch.from_numpy(heldV).to(torch.bfloat16).cuda(), 16, 64, 2)
    assert torch.equal(again, want)
