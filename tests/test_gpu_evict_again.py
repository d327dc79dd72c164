"""Eviction of the same sequences again and again on the GPU, against an oracle that keeps every
token's number (oracle/cache.py, evict_aged)."""
import numpy as np
import pytest

from oracle import cache as ocache
from tests.cache_cases import Pool

pytestmark = pytest.mark.gpu


def _held(pool, lens):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, T = len(lens), max(1, max(lens))
    p = mita.CacheParams(B, pool.Hkv, pool.Hkv, T, pool.d, pool.page, pool.n_pages, pool.cols, dtype=pool.p.dtype)
    ws = mita.cache_workspace(p)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    K, V = (torch.zeros((B, pool.Hkv, T, pool.d), dtype=pool.td, device="cuda") for _ in range(2))
    mita.mita_cache_read(p, pool.cache, pool.table, ln, K, V, ws, counts=ln)
    mita.mita_device_status(ws)
    return K.view(torch.int16), V.view(torch.int16)


def _sums(rng, n, kind):
    a = np.exp(2 * rng.standard_normal(n)).astype(np.float32)
    if kind == "ties":
        a = rng.integers(0, 3, n).astype(np.float32)
    elif kind == "special":
        pick = rng.random(n)
        a[pick < 0.1], a[(pick >= 0.1) & (pick < 0.2)], a[(pick >= 0.2) & (pick < 0.5)] = np.nan, np.inf, -np.inf
        a[(pick >= 0.5) & (pick < 0.6)] = -0.0
    return a


MANY = [1, 1, 64, 1, 300, 2, 0, 64, 64, 700, 5, 1, 1, 64]
CASES = [
    # d, page, Hkv, places, first lengths, keep, first, recents, tokens between calls, sums
    (64, 16, 2, 96, [40, 48, 70], [48, 48, 50], 2, [8], [1] * 20 + [5, 30, 1, 1], "any"),
    (128, 16, 3, 64, [10, 33], [20, 30], 0, [20, 3, 0, 20, 20], [1, 2, 3, 19, 20, 21, 1, 1, 1, 25, 1, 1], "ties"),
    (64, 32, 1, 512, [300, 300], [200, 260], 4, [196, 100], [1, 60, 9] * 5, "special"),        # nothing between stays
    (128, 64, 2, 4096, [2048, 3000], [2048, 2000], 4, [256], MANY, "any"),                     # one block a row
    (128, 48, 2, 4992, [2048, 4000], [2048, 3900], 4, [256, 256, 100], MANY, "any"),           # clusters of two,
    (64, 64, 2, 12288, [9001, 5000], [9000, 4000], 0, [512], MANY, "special"),                 # of four
    (128, 64, 1, 12288, [9001, 5000], [9000, 4000], 16, [333], MANY, "ties"),
    (64, 128, 2, 32768, [30000, 17000], [29000, 4096], 3, [1000, 1000, 64], MANY, "any"),      # and of eight
    (64, 128, 1, 400000, [396500], [395000], 5, [4000], [1, 600, 3000, 4000, 1, 77, 4100, 2, 1, 900, 1, 64], "any"),  # not held
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "d%d_p%d_H%d_n%d_%s" % (c[0], c[1], c[2], c[3], c[9]))
def test_eviction_again_matches_oracle(case):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    d, page, Hkv, cap, lens, keep, first, recents, overs, kind = case
    rng, B = np.random.default_rng(cap + d), len(lens)
    pool = Pool([cap] * B, Hkv, d, page, "bf16", seed=2)
    assert pool.cols * page == cap
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    ws, keep_t, n = mita.cache_evict_workspace(pool.p), i32(keep), list(lens)
    age = torch.zeros((B, Hkv, cap), dtype=torch.int32, device="cuda")
    sums = np.full((B, Hkv, cap), np.nan, np.float32)
    newest = list(n)
    born = [[np.arange(n[b]) for _ in range(Hkv)] for b in range(B)]
    for b in range(B):
        for h in range(Hkv):
            sums[b, h, :n[b]] = _sums(rng, n[b], kind)
    for turn, over in enumerate([0] + overs):
        recent = recents[turn % len(recents)]
        for b in range(B):
            c = min(over + b, cap - n[b])  # (the sequences' own)
            for h in range(Hkv):
                born[b][h] = np.r_[born[b][h], np.arange(newest[b], newest[b] + c)]
                sums[b, h, n[b]:n[b] + c] = 1e-4 * _sums(rng, c, kind)  # the young have little
                sums[b, h, :n[b]] *= np.float32(rng.uniform(0.5, 1.5))
            n[b], newest[b] = n[b] + c, newest[b] + c
        acc, ln = torch.from_numpy(sums).cuda(), i32(n)
        src = torch.full((B, Hkv, cap), -7, dtype=torch.int32, device="cuda")
        in_place = turn % 2 == 0
        acc_out = acc if in_place else torch.full_like(acc, 7.0)
        len_out = ln if in_place else i32([-7] * B)
        K0, V0 = _held(pool, n)
        ws.fill_(0xff)
        mita.mita_cache_evict(pool.p, pool.cache, pool.table, ln, keep_t, acc, ws, first=first, recent=recent,
                              len_out=len_out, acc_out=acc_out, src_out=src, age=age)
        mita.mita_device_status(ws)
        now = [min(x, k) for x, k in zip(n, keep)]
        assert len_out.tolist() == now
        K1, V1 = _held(pool, now)
        got, ages, places = acc_out.cpu().numpy(), age.cpu().numpy(), src.cpu().numpy()
        for b in range(B):
            for h in range(Hkv):
                want = ocache.evict_aged(sums[b, h, :n[b]], born[b][h], keep[b], first, recent, newest[b])
                assert np.array_equal(places[b, h, :now[b]], want), (turn, b, h)
                assert (places[b, h, now[b]:] == -7).all()
                at = torch.from_numpy(want.astype(np.int64)).cuda()
                assert torch.equal(K0[b, h][at], K1[b, h, :now[b]]) and torch.equal(V0[b, h][at], V1[b, h, :now[b]])
                old = sums[b, h].copy()
                sums[b, h, :now[b]] = old[want]
                tail = old[now[b]:] if in_place else np.full(cap - now[b], 7.0, np.float32)
                np.testing.assert_array_equal(got[b, h].view(np.int32), np.r_[old[want], tail].view(np.int32))
                born[b][h] = born[b][h][want]
                # an unmoved token at place p is newest - now + p
                assert np.array_equal(ages[b, h, :now[b]], np.arange(now[b]) - (born[b][h] - (newest[b] - now[b]))), (turn, b, h)
                assert not ages[b, h, now[b]:].any()
            n[b] = now[b]


def test_drafts_taken_back():
    """Tokens that are appended and taken back again (rejected drafts) leave nothing behind."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    rng, keep, recent, cap = np.random.default_rng(3), 60, 12, 128
    pool = Pool([cap], 2, 64, 16, "bf16", seed=2)
    ws, age = mita.cache_evict_workspace(pool.p), torch.zeros((1, 2, cap), dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor([x], dtype=torch.int32).cuda()
    n, newest = keep, keep
    born, sums = [np.arange(n) for _ in range(2)], rng.random((1, 2, cap)).astype(np.float32)
    for turn in range(16):
        took = int(rng.integers(1, 6))  # of six drafts
        born = [np.r_[x, np.arange(newest, newest + took)] for x in born]
        n, newest = n + took, newest + took
        sums[0, :, n - took:n] = 1e-6 * rng.random((2, took))
        sums[0, :, n:] = 1e6  # what the others left
        acc, ln, src = torch.from_numpy(sums).cuda(), i32(n), torch.zeros((1, 2, cap), dtype=torch.int32, device="cuda")
        mita.mita_cache_evict(pool.p, pool.cache, pool.table, ln, i32(keep), acc, ws, first=1, recent=recent, src_out=src, age=age)
        mita.mita_device_status(ws)
        for h in range(2):
            want = ocache.evict_aged(sums[0, h, :n], born[h], keep, 1, recent, newest)
            assert src[0, h, :keep].tolist() == want.tolist()
            born[h] = born[h][want]
            assert np.isin(np.arange(newest - recent, newest), born[h]).all()
        sums, n = acc.cpu().numpy(), keep


def test_ages_of_all_sizes_stay_in_bounds():
    """Numbers that no sequence of calls leaves choose some tokens, and move nothing out of range; ages end at 2^30."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    n, keep = 300, 100
    pool = Pool([n], 1, 64, 16, "bf16", seed=2)
    cap = pool.cols * 16
    for value in (2 ** 31 - 1, -2 ** 31, 2 ** 30, -5):
        ws, acc = mita.cache_evict_workspace(pool.p), torch.rand((1, 1, cap), device="cuda")
        age = torch.full((1, 1, cap), value, dtype=torch.int32, device="cuda")
        src = torch.full((1, 1, cap), -7, dtype=torch.int32, device="cuda")
        mita.mita_cache_evict(pool.p, pool.cache, pool.table, pool.len_t.clone(), torch.tensor([keep], dtype=torch.int32).cuda(),
                              acc, ws, first=2, recent=8, src_out=src, age=age)
        mita.mita_device_status(ws)
        kept = src[0, 0, :keep].tolist()
        assert len(set(kept)) == keep and min(kept) >= 0 and max(kept) < n
        assert int(age[..., :keep].max()) <= 2 ** 30 and int(age[..., :keep].min()) >= -2 ** 30 and not age[0, 0, keep:n].any()
        assert (age[0, 0, n:] == value).all()


def test_decoding_loop_keeps_the_newest():
    """Store, attend, weigh and evict in one graph, one token a turn: the newest tokens stay, in every head and turn."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, H, Hkv, d, page, budget, first, recent, cols = 3, 8, 2, 64, 16, 48, 2, 8, 6
    start, cap = [40, 48, 10], cols * page
    gen = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    table = torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols)
    p = mita.CacheParams(B, H, Hkv, 1, d, page, B * cols, cols, flags=mita.FLAG_CAUSAL)
    fill = mita.CacheParams(B, Hkv, Hkv, max(start), d, page, B * cols, cols)
    cache, lens = torch.zeros(mita.mita_cache_size(p), dtype=torch.uint8, device="cuda"), i32(start)
    mita.mita_cache_write(fill, rnd(B, Hkv, max(start), d), rnd(B, Hkv, max(start), d), cache, table, lens,
                          mita.cache_workspace(fill), counts=lens)
    acc, weighed = torch.rand((B, Hkv, cap), generator=gen).cuda(), torch.zeros((B, Hkv, cap), device="cuda")
    age, src = (torch.zeros((B, Hkv, cap), dtype=torch.int32, device="cuda") for _ in range(2))
    ws, ews = mita.cache_workspace(p), mita.cache_evict_workspace(p)
    Q, K, V, O = rnd(B, H, 1, d), rnd(B, Hkv, 1, d), rnd(B, Hkv, 1, d), rnd(B, H, 1, d)
    lse, keep = torch.zeros((B, H, 1), device="cuda"), i32([budget] * B)

    def step():
        lens.add_(1)
        mita.mita_cache_write(p, K, V, cache, table, lens, ws)
        mita.mita_cache_attention(p, Q, cache, table, lens, O, ws, lse_out=lse)
        mita.mita_cache_weights(p, Q, cache, table, lens, lse, acc, ws, decay=0.9, acc_out=weighed)
        mita.mita_cache_evict(p, cache, table, lens, keep, weighed, ews, first=first, recent=recent, acc_out=acc, src_out=src, age=age)

    was = [t.clone() for t in (cache, lens, acc, age)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # the modules load outside of the capture
    torch.cuda.synchronize()
    for t, w in zip((cache, lens, acc, age), was):
        t.copy_(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    born = [[np.arange(x) for _ in range(Hkv)] for x in start]
    newest, n = list(start), list(start)
    for _ in range(40):
        for x in (Q, K, V):
            x.copy_(rnd(*x.shape))
        graph.replay()
        mita.mita_device_status(ews)
        for b in range(B):
            n[b], newest[b] = n[b] + 1, newest[b] + 1
            for h in range(Hkv):
                born[b][h] = np.r_[born[b][h], newest[b] - 1]
                want = ocache.evict_aged(weighed[b, h, :n[b]].cpu().numpy(), born[b][h], budget, first, recent, newest[b])
                assert src[b, h, :len(want)].tolist() == want.tolist()
                born[b][h] = born[b][h][want]
                assert np.isin(np.arange(newest[b] - recent, newest[b]), born[b][h]).all()
            n[b] = min(n[b], budget)


@pytest.mark.parametrize("odd_acc,odd_age", [(False, True), (True, False), (True, True)])
def test_ages_aligned_to_their_elements(odd_acc, odd_age):
    """Sums or ages that are aligned to their elements only give what aligned ones give, on another stream too."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    lens, keep, shape = [4997, 300], [1234, 200], (2, 2, 5008)
    pool = Pool(lens, 2, 64, 16, "bf16", seed=3)
    cap = pool.cols * 16
    assert cap == shape[2]
    rng = np.random.default_rng(6)
    sums, start = _sums(rng, shape, "any"), rng.integers(-300, 300, shape).astype(np.int32)
    for b, n in enumerate(lens):
        start[b, :, n:] = 0

    def run(odd_acc, odd_age, stream):
        place = lambda x, odd: torch.cat([torch.zeros(int(odd), dtype=x.dtype), x.flatten()]).cuda()[int(odd):].view(x.shape)
        acc, age = place(torch.from_numpy(sums), odd_acc), place(torch.from_numpy(start), odd_age)
        out, src, new = torch.zeros_like(acc), torch.zeros(shape, dtype=torch.int32, device="cuda"), torch.zeros_like(pool.len_t)
        ws, cache = mita.cache_evict_workspace(pool.p), pool.cache.clone()
        kp = torch.tensor(keep, dtype=torch.int32).cuda()
        torch.cuda.synchronize()
        mita.mita_cache_evict(pool.p, cache, pool.table, pool.len_t, kp, acc, ws, first=1, recent=64, len_out=new, acc_out=out,
                              src_out=src, age=age, stream=stream)
        mita.mita_device_status(ws, stream)
        return out, src, new, cache, age

    for a, b in zip(run(False, False, None), run(odd_acc, odd_age, torch.cuda.Stream())):
        assert torch.equal(a, b)
