"""Failure detection of the cached tokens' weights, tested without a GPU fault.

Every wait of the tiles on tcgen05 is bounded. With MITA_TESTFLAG_STALL_PRODUCER one block
waits for one signal more than comes, and waits give up after about a millisecond. The call must report
MITA_ERR_TIMEOUT, and the next ordinary call on the same workspace must be the same bits as before.
"""
import pytest

from tests.cache_cases import Pool

pytestmark = pytest.mark.gpu

# dtype, d, query heads a cache head, T: one tile of up to 64 rows, several of 128, several passes
FORMS = [("bf16", 128, 6, 5), ("bf16", 64, 40, 1), ("bf16", 128, 64, 4), ("f32", 128, 20, 1), ("f32", 64, 90, 7)]
LENS = {"short": [100], "long": [20000], "many": [130] * 700}


@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "%s_d%d_G%d_T%d" % f)
def test_stalled_weights_time_out_then_recover(form, lens):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    dtype, d, G, T = form
    pool = Pool(LENS[lens], 1, d, 64, dtype, seed=d)
    B = len(LENS[lens])
    p = [mita.CacheParams(B, G, 1, T, d, 64, pool.n_pages, pool.cols, 0.0, mita.FLAG_CAUSAL | f, pool.p.dtype)
         for f in (0, mita.TESTFLAG_STALL_PRODUCER)]
    ws = mita.cache_workspace(p[0])
    gen = torch.Generator().manual_seed(1)
    Q = torch.randn((B, G, T, d), generator=gen).to(pool.td).cuda()
    lse = torch.full((B, G, T), 6.0, device="cuda")

    def call(which):
        out = torch.zeros((B, 1, pool.cols * 64), device="cuda")
        mita.mita_cache_weights(p[which], Q, pool.cache, pool.table, pool.len_t, lse, None, ws, decay=0.0, acc_out=out)
        return out

    want = call(0)
    mita.mita_device_status(ws)
    assert want.any()
    for _ in range(2):
        call(1)
        with pytest.raises(mita.MitaError) as err:
            mita.mita_device_status(ws)
        assert err.value.status == 5, err.value  # MITA_ERR_TIMEOUT
        mita.mita_device_status(ws)  # reading the word cleared it
    for _ in range(2):
        assert torch.equal(call(0), want)
        mita.mita_device_status(ws)
