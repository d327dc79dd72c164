"""Pins of the 4-bit cache's oracle (no GPU): the two grids, the rounding of
ties and quotients, and attention against plain softmax attention."""
import numpy as np
import pytest
import torch

from oracle import cache as oc


def test_scales_are_torch_e4m3():
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(bits, oc.E4M3)
    x = np.abs(np.random.default_rng(0).standard_normal(20000) * np.exp(np.random.default_rng(1).uniform(-7, 5, 20000)))
    x = np.minimum(x.astype(np.float32), 448.0)
    mid = ((oc.E4M3[1:] + oc.E4M3[:-1]) / 2).astype(np.float32)  # exact ties
    for a in (x, mid):
        want = torch.from_numpy(a).to(torch.float8_e4m3fn).double().numpy()
        np.testing.assert_array_equal(oc.nearest(a, oc.E4M3), want)


def test_codes_by_brute_force():
    a = np.concatenate([np.linspace(0, 8, 4001), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]])
    got = oc.nearest(a, oc.E2M1)
    for x, g in zip(a, got):
        d = np.abs(oc.E2M1 - x)
        best = np.flatnonzero(d == d.min())
        assert g == oc.E2M1[best[best % 2 == 0][0] if len(best) > 1 else best[0]]
    assert list(got[-7:]) == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fp32_quotients_round_to_the_same_codes(dtype):
    """The correctly rounded fp32 quotient lands on a midpoint of the code grid
    only where the exact quotient does, so rounding either gives one code."""
    rng = np.random.default_rng(3)
    s = rng.choice(oc.E4M3[1:], 400000).astype(np.float32)
    y = (s * rng.choice(np.float32([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), s.size)).astype(np.float32)
    steps = rng.integers(-2, 3, s.size)  # at a midpoint and next to it
    bits = y.view(np.int32) + (steps << 16 if dtype == "bf16" else steps)
    y = bits.astype(np.int32).view(np.float32)
    exact = oc.nearest(y.astype(np.float64) / s, oc.E2M1)
    np.testing.assert_array_equal(oc.nearest((y / s).astype(np.float64), oc.E2M1), exact)


def test_fp32_scales_round_as_the_exact_quotient():
    """The correctly rounded fp32 quotient max / 6 is on a midpoint of the scales only
    where the exact quotient is: every midpoint and the floats next to 6 times it. A
    product by the rounded 1 / 6 is not enough: it moves some of them onto a midpoint."""
    mid = (oc.E4M3[1:] + oc.E4M3[:-1]) / 2
    a = (6 * mid).astype(np.float32)  # exact: 5 and 2 significant bits
    a = (a.view(np.int32)[:, None] + np.arange(-4, 5, dtype=np.int32)).view(np.float32).ravel()
    want = oc.nearest(a.astype(np.float64) / 6, oc.E4M3)
    np.testing.assert_array_equal(oc.nearest((a / np.float32(6)).astype(np.float64), oc.E4M3), want)
    product = oc.nearest((a * (np.float32(1) / np.float32(6))).astype(np.float64), oc.E4M3)
    assert 0 < int((product != want).sum()) < 40


def test_special_blocks():
    x = np.zeros((6, 16))
    x[1, 3], x[2, 4], x[3, 0] = np.nan, -np.inf, 1e30
    x[4] = 1e-6
    x[5] = np.arange(16) - 8.0
    v = oc.quantise(x)
    assert np.all(v[0] == 0) and np.all(np.isnan(v[1])) and np.all(v[4] == 0)
    assert v[2, 4] == -2688 and np.all(np.delete(v[2], 4) == 0) and v[3, 0] == 2688
    assert v[5, 8] == 0 and abs(v[5, 0] + 8) <= 8 / 12 + 8 / 16
    np.testing.assert_array_equal(oc.quantise(x[5] * 2.0 ** 30, 30), oc.quantise(x[5]) * 2.0 ** 30)


def test_quantisation_error_is_bounded():
    """Within half a code step of the block's scale everywhere the scale is a
    normal e4m3 number: |x - v| <= s, and 6 s >= amax / (1 + 2^-4)."""
    x = np.random.default_rng(5).standard_normal((1000, 64)) * 3
    v = oc.quantise(x)
    amax = np.abs(x.reshape(1000, 4, 16)).max(-1, keepdims=True)
    err = np.abs(x - v).reshape(1000, 4, 16)
    assert np.all(err <= amax / 6 * (1 + 2.0 ** -4))


def test_attention_is_softmax_attention():
    rng = np.random.default_rng(7)
    q, k, v = (torch.from_numpy(rng.standard_normal((n, 64))) for n in (5, 33, 33))
    lim = [33, 1, 17, 0, 32]
    o, lse, spread = oc.attention(q.numpy(), k.numpy(), v.numpy(), lim, 0.125)
    for r, m in enumerate(lim):
        if m == 0:
            assert np.all(o[r] == 0) and lse[r] == -np.inf
            continue
        want = torch.nn.functional.scaled_dot_product_attention(q[None, r:r + 1], k[None, :m], v[None, :m], scale=0.125)
        np.testing.assert_allclose(o[r], want[0, 0].numpy(), rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(lse[r], torch.logsumexp(k[:m] @ q[r] * 0.125, 0).item(), rtol=1e-12)
        assert np.all(spread[r] >= np.abs(o[r]) - 1e-15)
