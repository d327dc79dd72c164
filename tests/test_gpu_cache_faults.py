"""Failure detection of the cache attention, tested without a GPU fault.

Every wait of its tensor-core kernels is bounded. With
MITA_TESTFLAG_STALL_PRODUCER one warp of the register form, or one block of the
tiles on tcgen05, waits for one signal more than comes, and waits give up after about
a millisecond. The call must report MITA_ERR_TIMEOUT, with work left in the block's
piece or none, and the next ordinary call on the same workspace must be the same bits
as before: copies and products have landed and tensor memory is free again.
"""
import pytest

from tests.cache_cases import Pool

pytestmark = pytest.mark.gpu

# dtype, d, query heads a cache head, T: rows of a tile 8, 8, 16, 32, 64, 64, and float32's 8 and 16
FORMS = [("bf16", 128, 1, 1), ("bf16", 64, 1, 5), ("bf16", 128, 6, 2), ("bf16", 64, 3, 10), ("bf16", 128, 32, 2),
         ("bf16", 128, 5, 40), ("f32", 128, 1, 1), ("f32", 64, 6, 3)]
# one long sequence is cut over all blocks; of many short ones a block has several
LENS = {"short": [100], "long": [40000], "many": [130] * 1300}


def _calls(form, lens, flags):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    dtype, d, G, T = form
    pool = Pool(lens, 1, d, 64, dtype, seed=d)
    B = len(lens)
    p = [mita.CacheParams(B, G, 1, T, d, 64, pool.n_pages, pool.cols, 0.0, mita.FLAG_CAUSAL | f, pool.p.dtype)
         for f in (0, flags)]
    ws = mita.cache_workspace(p[0])
    assert mita.mita_cache_workspace_size(p[1]) <= ws.numel()
    Q = torch.randn((B, G, T, d), generator=torch.Generator().manual_seed(1)).to(pool.td).cuda()

    def call(which):
        O, L = torch.zeros_like(Q), torch.zeros((B, G, T), device="cuda")
        mita.mita_cache_attention(p[which], Q, pool.cache, pool.table, pool.len_t, O, ws, lse_out=L)
        return O, L

    return mita, ws, call


@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "%s_d%d_G%d_T%d" % f)
def test_stalled_attention_times_out_then_recovers(form, lens):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    mita, ws, call = _calls(form, LENS[lens], mita.TESTFLAG_STALL_PRODUCER)
    O, L = call(0)
    mita.mita_device_status(ws)
    for _ in range(2):
        call(1)
        with pytest.raises(mita.MitaError) as err:
            mita.mita_device_status(ws)
        assert err.value.status == 5, err.value  # MITA_ERR_TIMEOUT
        mita.mita_device_status(ws)  # reading the word cleared it
    for _ in range(2):
        O2, L2 = call(0)
        mita.mita_device_status(ws)
        assert torch.equal(O, O2) and torch.equal(L, L2)


def test_stall_flag_is_inert_on_cuda_cores():
    import torch
    import compressed_attention_adaptive_gb300 as mita
    mita, ws, call = _calls(FORMS[0], [300, 20], mita.FLAG_SIMT | mita.TESTFLAG_STALL_PRODUCER)
    O, _ = call(0)
    O2, _ = call(1)
    mita.mita_device_status(ws)
    assert torch.allclose(O.float(), O2.float(), rtol=2 ** -6, atol=2 ** -8)
