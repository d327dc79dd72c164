"""Rotation at the farthest positions, by frequencies of either sign and any size, against the
oracle (oracle/rope.py)."""
import numpy as np
import pytest

from oracle import rope as orope

pytestmark = pytest.mark.gpu


def _freqs(kind, n):
    if kind == "usual":
        return 10000.0 ** (-np.arange(n) / n)
    if kind == "negated":
        return -(10000.0 ** (-np.arange(n) / n))
    rng = np.random.default_rng(5)
    f = rng.uniform(-1, 1, n) * 2.0 ** rng.integers(-30, 21, n)
    f[:4] = 0.0, 1e6, -1e6, -2.0 ** -60
    return f


@pytest.mark.parametrize("back", [False, True], ids=["", "back"])
@pytest.mark.parametrize("kind", ["usual", "negated", "mixed"])
def test_far_positions_lose_nothing(kind, back):
    """|gpu - oracle| of float32 rows, of |x0| + |x1|:
      - the angle's float: half a step of at most 1/2 turn, 2^-25 half turns, pi times: 0.8 2^-23;
      - sincospi 2^-22, its products, their sum and the output: 4 2^-24 (|y| <= |x0| + |x1|): 4 2^-23 in all;
      - the frequency in turns: at most 2^-63 of a turn and 2^-104 of itself for each position, 2^-29 at
        most for 2^31 of them, and 2^-50 for angles of 2^51.
    5 2^-23 covers all."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    d, T = 128, 400
    f = _freqs(kind, d // 2)
    rng = np.random.default_rng(8)
    pos = np.r_[rng.integers(-2 ** 31, 2 ** 31, T - 4), [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -3]]
    p = mita.RopeParams(1, 2, 0, T, d, d, freqs=tuple(f), dtype=mita.F32)
    x = torch.randn((1, 2, T, d), generator=torch.Generator().manual_seed(2)).cuda()
    y = torch.empty_like(x)
    (mita.mita_rope_backward if back else mita.mita_rope)(p, x, None, y, None, pos=torch.from_numpy(pos.astype(np.int32)).cuda())
    xn, got = x.double().cpu().numpy(), y.double().cpu().numpy()
    want = orope.rotate(xn, pos, f, d, back=back)
    size = np.abs(xn[..., :d // 2]) + np.abs(xn[..., d // 2:])
    worst = float((np.abs(got - want) / np.concatenate([size, size], -1)).max()) * 2.0 ** 23
    assert worst <= 5, worst
