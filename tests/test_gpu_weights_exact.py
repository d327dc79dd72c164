"""What float32 rows' lower halves add to a score of the cached tokens' weights, on the GPU: sums are cut to 24
bits at every step, so that they have to be added up before the upper halves, or apart from them."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,rows,tile", [(128, 1, False), (128, 2, False), (128, 3, False), (128, 8, False), (128, 9, True),
                                         (128, 64, True), (128, 65, True), (128, 300, True), (64, 1, False), (64, 2, False),
                                         (64, 7, False), (64, 16, False), (64, 32, False), (64, 33, True), (64, 200, True)])
def test_lower_halves_count(d, rows, tile):
    """A row of 64 in one channel and 1 + 15 2^-23 in 14 others of its block, zeros elsewhere; keys of 1. The upper halves' sum
    is 78, exactly, in any order, and its 24 bits end at 2^-17. The lower halves are 15 2^-23 each, four of them in a step less than
    that, 3.3 times it in all: a sum that takes them in behind the 64 loses all of them, 1.25e-5 of the weight at a scale of 1/2.
      - In a sum of their own they are exact, and the two sums' sum is off by half a step: 2^-18, 2^-19 of the weight.
      - Before the others in the same sum (tiles) less than a whole step is lost when 64 comes, and nothing then: 2^-18.
      - The difference to the log sum is -3/4, off by 2^-25; log2(e) and its product 2^-24 each, the exponential 2^-22: below 2^-21.
    All rows but one have an infinite log sum and add nothing."""
    import compressed_attention_adaptive_gb300 as mita
    n, page = 300, 32
    cols = -(-n // page)
    p = mita.CacheParams(1, rows, 1, 1, d, page, cols, cols, scale=0.5, dtype=mita.F32)
    w = mita.CacheParams(1, 1, 1, n, d, page, cols, cols, dtype=mita.F32)
    K = torch.ones((1, 1, n, d), device="cuda")
    K[..., ::16] = 6.0  # scales of 1
    cache = torch.zeros(mita.mita_cache_size(p), dtype=torch.uint8, device="cuda")
    table, lens = torch.arange(cols, dtype=torch.int32, device="cuda").view(1, cols), torch.tensor([n], dtype=torch.int32).cuda()
    ws = mita.cache_workspace(w)
    mita.mita_cache_write(w, K, K, cache, table, lens, ws)
    mita.mita_device_status(ws)
    want = math.exp(0.5 * (64 + 14 * (1 + 15 * 2.0 ** -23)) - 39.75)
    ws = mita.cache_workspace(p)
    for block in range(0, d, 16):
        q = np.zeros(d, np.float32)
        q[block + 1], q[block + 2:block + 16] = 64, 1 + 15 * 2.0 ** -23
        for r in sorted({0, rows // 2, rows - 1}):
            lse, Q = torch.full((1, rows, 1), math.inf, device="cuda"), torch.zeros((1, rows, 1, d), device="cuda")
            lse[0, r], Q[0, r, 0] = 39.75, torch.from_numpy(q).cuda()
            out = torch.zeros((1, 1, cols * page), device="cuda")
            mita.mita_cache_weights(p, Q, cache, table, lens, lse, None, ws, decay=0.0, acc_out=out)
            mita.mita_device_status(ws)
            off = float((out[0, 0, :n].double() / want - 1).abs().max())
            assert off <= (2.0 ** -18 if tile else 2.0 ** -19) + 2.0 ** -21, (block, r, off)
