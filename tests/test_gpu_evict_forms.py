"""Eviction and cached tokens' weights in forms and with faults that the other tests do not come to: clusters of
four, rows too long for shared memory, one block for each of many rows; what is right beside what is out of range."""
import numpy as np
import pytest
import torch

from oracle import cache as ocache

pytestmark = pytest.mark.gpu


def _sums(rng, shape, kind):
    a = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        a = rng.integers(0, 4, shape).astype(np.float32)
    elif kind == "special":
        pick = rng.random(shape)
        a[pick < 0.1], a[(pick >= 0.1) & (pick < 0.3)], a[(pick >= 0.3) & (pick < 0.4)] = np.nan, np.inf, -np.inf
        a[(pick >= 0.4) & (pick < 0.7)], a[(pick >= 0.7) & (pick < 0.9)] = -0.0, 0.0
    return a


@pytest.mark.parametrize("d,page,Hkv,lens,keep,first,recent,kind", [
    (64, 16, 2, [9001, 5000], [3000, 4999], 4, 64, "any"),        # clusters of four
    (128, 64, 2, [9001, 5000], [3000, 20], 0, 0, "ties"),
    (128, 32, 3, [16000, 12345], [8000, 12000], 7, 333, "special"),
    (64, 64, 1, [400000], [150000], 3, 20, "any"),                # too long to hold, in clusters of eight
    (64, 64, 1, [393300], [100], 3, 20, "special"),
    (64, 64, 160, [52000], [20000], 4, 256, "any"),               # and by one block each
    (64, 64, 160, [50003], [49000], 0, 3, "ties"),
])
def test_forms_match_oracle(d, page, Hkv, lens, keep, first, recent, kind):
    import compressed_attention_adaptive_gb300 as mita
    rng, B = np.random.default_rng(d + Hkv), len(lens)
    need = [-(-n // page) for n in lens]
    cols, n_pages = max(need), sum(need)
    cap = cols * page
    p = mita.CacheParams(B, Hkv, Hkv, 1, d, page, n_pages, cols)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randint(0, 256, (mita.mita_cache_size(p),), dtype=torch.uint8, device="cuda", generator=g)
    table, perm, at = np.zeros((B, cols), np.int32), rng.permutation(n_pages), 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
    table, ln, kp = i32(table), i32(lens), i32(keep)
    rp = mita.CacheParams(B, Hkv, Hkv, max(lens), d, page, n_pages, cols)
    rows = torch.zeros((2, B, Hkv, max(lens), d), dtype=torch.bfloat16, device="cuda")
    got = torch.zeros_like(rows)
    rws, ws = mita.cache_workspace(rp), mita.cache_evict_workspace(p)
    mita.mita_cache_read(rp, cache, table, ln, rows[0], rows[1], rws, counts=ln)
    sums = _sums(rng, (B, Hkv, cap), kind)
    acc = torch.from_numpy(sums).cuda()
    src = torch.full(acc.shape, -7, dtype=torch.int32, device="cuda")
    new = torch.zeros_like(ln)
    mita.mita_cache_evict(p, cache, table, ln, kp, acc, ws, first=first, recent=recent, len_out=new, src_out=src)
    mita.mita_device_status(ws)
    mita.mita_cache_read(rp, cache, table, ln, got[0], got[1], rws, counts=ln)
    mita.mita_device_status(rws)
    assert new.tolist() == keep
    for b in range(B):
        heads = range(Hkv) if Hkv < 8 else sorted({0, Hkv - 1, *rng.integers(0, Hkv, 4).tolist()})
        for h in heads:
            want = ocache.evict(sums[b, h, :lens[b]], keep[b], first, recent)
            assert np.array_equal(src[b, h, :keep[b]].cpu().numpy(), want), (b, h)
            np.testing.assert_array_equal(acc[b, h, :keep[b]].cpu().numpy().view(np.int32), sums[b, h][want].view(np.int32))
        at = src[b, :, :keep[b]].long()[None, :, :, None].expand(2, -1, -1, d)
        moved = torch.gather(rows[:, b], 2, at)
        assert torch.equal(got[:, b, :, :keep[b]].view(torch.int16), moved.view(torch.int16))
        assert torch.equal(got[:, b, :, keep[b]:].view(torch.int16), rows[:, b, :, keep[b]:].view(torch.int16))


@pytest.mark.parametrize("dtype,H,T,simt", [("bf16", 2, 1, False), ("bf16", 6, 1, False), ("bf16", 40, 2, False), ("f32", 6, 2, False),
                                            ("f32", 40, 2, False), ("bf16", 6, 1, True), ("f32", 40, 2, True)])
def test_sums_beside_bad_lengths_and_exponents(dtype, H, T, simt):
    """A length out of range is reported and leaves the other sequences' sums as they should be, an exponent the other heads'."""
    import compressed_attention_adaptive_gb300 as mita
    from tests.cache_cases import Pool
    lens = [300, 200, 129]
    pool = Pool(lens, 2, 128, 32, dtype, seed=8)
    for b in range(3):  # every entry names a page
        pool.table[b, -(-lens[b] // 32):] = b
    p = mita.CacheParams(3, H, 2, T, 128, 32, pool.n_pages, pool.cols, flags=mita.FLAG_SIMT if simt else 0, dtype=pool.p.dtype)
    gen = torch.Generator().manual_seed(4)
    Q, lse = torch.randn((3, H, T, 128), generator=gen).to(pool.td).cuda(), torch.full((3, H, T), 7.0, device="cuda")
    acc = torch.rand((3, 2, pool.cols * 32), generator=gen).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()

    def run(ln, exps, status):
        out, ws = torch.full_like(acc, 7.0), mita.cache_workspace(p)
        mita.mita_cache_weights(p, Q, pool.cache, pool.table, ln, lse, acc, ws, exps=exps, acc_out=out)
        if status:
            with pytest.raises(mita.MitaError) as e:
                mita.mita_device_status(ws)
            assert e.value.status == status
            del e  # (holds this frame)
        mita.mita_device_status(ws)
        return out

    want = run(pool.len_t, None, 0)
    assert (want[1, :, 200:] == 7.0).all() and not (want[1, :, :200] == 7.0).any()
    for n in (-1, -2 ** 31, pool.cols * 32 + 1, 2 ** 31 - 1):
        out = run(i32(300, n, 129), None, 6)
        assert torch.equal(out[[0, 2]], want[[0, 2]])
        assert n > 0 or (out[1] == 7.0).all()
    for e in (61, -61, 2 ** 31 - 1, -2 ** 31):
        for exps, head in ((i32(0, e, 0, 0), 0), (i32(e, 0, 0, 0), 1)):
            out = run(pool.len_t, exps.view(2, 2), 6)
            assert torch.equal(out[:, head], want[:, head])
        out = run(pool.len_t, i32(0, 0, 0, e).view(2, 2), 6)  # the values' have no part in the sums
        assert torch.equal(out, want)
