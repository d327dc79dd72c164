"""Rotary positions on the GPU against the oracle (oracle/rope.py)."""
import numpy as np
import pytest

from oracle import rope as orope
from tests import parity

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _bound(dtype, x, y, pos, freqs, rot, interleaved, gain):
    """Allowed |gpu - oracle|, u half a step of the output's type (bf16 2^-8, float 2^-24):
      - the output's rounding: u |y|;
      - the angle: its float has 2^-24 of at most pi (1.6 2^-23), the frequency in turns and the
        position's product with it 2^-52 of the whole angle;
      - sincospi's own error, at most 2^-22 of a number up to 1, and the rounding of its product with
        the gain and of the gain, 2^-24 each;
      - two products and a sum: 3 2^-24,
    the last three lines of |gain| (|x0| + |x1|): 2 + 2 + 2 steps of 2^-23, so 6."""
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    p, q = orope.pairs(rot, interleaved)
    b = np.abs(y) * u
    far = np.abs(np.asarray(pos, np.float64))[..., None] * np.abs(np.asarray(freqs, np.float64)) * 2.0 ** -51
    each = abs(gain) * (np.abs(x[..., p]) + np.abs(x[..., q])) * (6 * 2.0 ** -23 + far)
    b[..., p] += each
    b[..., q] += each
    b[..., rot:] = 0  # copied
    return b


def _check(dtype, x, got, pos, freqs, rot, interleaved, gain, back, label):
    x, got = _np(x), _np(got)
    y = orope.rotate(x, pos, freqs, rot, interleaved, gain, back)
    bound = _bound(dtype, x, y, pos, freqs, rot, interleaved, gain)
    diff = np.abs(got - y)
    assert np.all(diff <= bound), (label, float((diff / np.maximum(bound, 1e-300)).max()))
    parity.REPORT.append(("rope " + label, float((diff[..., :rot] / np.maximum(bound[..., :rot], 1e-300)).max()), 0.0, y.size))


def _rows(B, H, T, d, td, seed, source):
    """[B, H, T, d] contiguous, or seen through a projection's [B, T, H + 3, d], or with odd strides."""
    import torch
    g = torch.Generator().manual_seed(seed)
    if source == "heads":
        return torch.randn((B, H, T, d), generator=g).to(td).cuda()
    if source == "proj":
        return torch.randn((B, T, H + 3, d), generator=g).to(td).cuda().transpose(1, 2)[:, 2:2 + H]
    if source == "odd":  # every row one element off a multiple
        return torch.randn((B, H, T, d + 1), generator=g).to(td).cuda()[..., 1:]
    return torch.randn((1, H, 1, d), generator=g).to(td).cuda().expand(B, H, T, d)  # repeated rows


CASES = [
    # dtype, B, H, Hkv, T, d, rot, interleaved, source, gain
    ("bf16", 1, 1, 1, 1, 128, 128, False, "heads", 0.0),
    ("bf16", 3, 5, 2, 33, 128, 128, False, "proj", 1.25),
    ("bf16", 2, 4, 4, 130, 64, 32, True, "proj", 0.0),
    ("bf16", 2, 3, 1, 7, 80, 20, False, "heads", 0.0),     # 10 pairs: two at a time
    ("bf16", 2, 3, 1, 7, 80, 20, True, "heads", 0.0),
    ("bf16", 1, 2, 2, 65, 72, 18, False, "heads", 0.5),    # 9 pairs: one at a time
    ("bf16", 1, 2, 1, 9, 256, 256, True, "odd", 0.0),
    ("bf16", 2, 2, 1, 5, 256, 2, False, "heads", 0.0),     # one pair, the rest copied
    ("bf16", 1, 1, 1, 3, 2, 2, True, "heads", 0.0),
    ("f32", 2, 7, 1, 50, 64, 64, False, "proj", 0.0),
    ("f32", 1, 3, 3, 11, 80, 20, True, "heads", 1.0),
    ("f32", 2, 2, 2, 4, 6, 4, False, "odd", -2.0),
    ("f32", 3, 1, 1, 260, 128, 96, True, "repeat", 0.0),
    ("f32", 1, 40, 8, 1, 128, 128, False, "repeat", 0.0),
    ("bf16", 1, 3, 0, 12, 64, 64, False, "heads", 0.0),    # queries alone
    ("bf16", 2, 300, 1, 600, 64, 64, False, "proj", 0.0),  # blocks over many heads
]


@pytest.mark.parametrize("back", [False, True], ids=["", "back"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_B%d_H%d_%d_T%d_d%d_r%d_%d_%s" % c[:9])
def test_rope_matches_oracle(case, back):
    import torch
    import compressed_attention_adaptive_gb300 as mita
    dtype, B, H, Hkv, T, d, rot, il, source, gain = case
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    freqs = mita.mita_rope_frequencies(rot)
    p = mita.RopeParams(B, H, Hkv, T, d, rot, None, gain, mita.FLAG_INTERLEAVED * il, mita.BF16 if dtype == "bf16" else mita.F32)
    Q, K = _rows(B, H, T, d, td, 1, source), _rows(B, Hkv, T, d, td, 2, source) if Hkv else None
    rng = np.random.default_rng(T)
    for name, pos in (("none", None), ("own", rng.integers(-500, 200000, (B, T))), ("shared", rng.integers(0, 4000, T)),
                      ("far", rng.integers(-2 ** 31, 2 ** 31, (B, T)))):
        Qo = torch.full((B, H, T, d), 7.0, dtype=td, device="cuda")
        Ko = torch.full((B, Hkv, T, d), 7.0, dtype=td, device="cuda") if Hkv else None
        pt = None if pos is None else torch.from_numpy(pos.astype(np.int32)).cuda()
        (mita.mita_rope_backward if back else mita.mita_rope)(p, Q, K, Qo, Ko, pos=pt)
        at = np.broadcast_to(np.arange(T) if pos is None else pos, (B, T))[:, None]
        for x, y in ((Q, Qo), (K, Ko)):
            if x is not None:
                _check(dtype, x, y, at, freqs, rot, il, gain or 1.0, back, "%s d%d/%d %s" % (dtype, rot, d, name))


@pytest.mark.parametrize("dtype,d,rot,il", [("bf16", 128, 128, False), ("f32", 64, 32, True), ("bf16", 72, 18, False)])
def test_in_place_inside_a_projection(dtype, d, rot, il):
    """Q and K rotated where they are, in one buffer with V: the same bits as elsewhere, V and the
    buffer's other elements untouched."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, H, Hkv, T = 2, 4, 2, 19
    p = mita.RopeParams(B, H, Hkv, T, d, rot, flags=mita.FLAG_INTERLEAVED * il, dtype=mita.BF16 if dtype == "bf16" else mita.F32)
    both = torch.randn((B, T, H + 2 * Hkv, d), generator=torch.Generator().manual_seed(0)).to(td).cuda()
    rows = both.transpose(1, 2)
    want = [torch.empty((B, h, T, d), dtype=td, device="cuda") for h in (H, Hkv)]
    mita.mita_rope(p, rows[:, :H], rows[:, H:H + Hkv], *want)
    before = both.clone()
    q, k = rows[:, :H], rows[:, H:H + Hkv]
    mita.mita_rope(p, q, k, q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(rows[:, H + Hkv:], before.transpose(1, 2)[:, H + Hkv:])
    # into a projection-shaped buffer of their own, next to each other
    out = torch.full((B, T, H + Hkv, d), 7.0, dtype=td, device="cuda").transpose(1, 2)
    r0 = before.transpose(1, 2)
    mita.mita_rope(p, r0[:, :H], r0[:, H:H + Hkv], out[:, :H], out[:, H:])
    assert torch.equal(out[:, :H], want[0]) and torch.equal(out[:, H:], want[1])
    # a view with other strides over the same memory is refused
    with pytest.raises(mita.MitaError):
        mita.mita_rope(p, rows[:, :H], rows[:, H:H + Hkv], rows[:, 1:1 + H], want[1])


def test_position_zero_and_special_numbers():
    import torch
    import compressed_attention_adaptive_gb300 as mita
    p = mita.RopeParams(1, 1, 0, 3, 64, 32)
    x = torch.randn((1, 1, 3, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    x[0, 0, 1, 5], x[0, 0, 1, 60], x[0, 0, 2, 40] = float("nan"), float("inf"), float("-inf")
    y = torch.empty_like(x)
    mita.mita_rope(p, x, None, y, None, pos=torch.tensor([0, 3, 9], dtype=torch.int32).cuda())
    assert torch.equal(y[0, 0, 0], x[0, 0, 0])
    bad = y[0, 0, 1].isnan()
    assert bad[5] and bad[21] and int(bad.sum()) == 2  # its own pair
    assert y[0, 0, 1, 60] == float("inf") and y[0, 0, 2, 40] == float("-inf")


@pytest.mark.parametrize("dtype,il,rot", [("f32", False, 64), ("f32", True, 20)])
def test_backward_is_the_gradient(dtype, il, rot):
    """Against differences of the forward pass, and as its transpose: <g, R x> = <R^T g, x>."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, H, T, d = 2, 2, 5, 64
    p = mita.RopeParams(B, H, 0, T, d, rot, gain=1.3, flags=mita.FLAG_INTERLEAVED * il, dtype=mita.F32)
    gen = torch.Generator().manual_seed(4)
    x, g = (torch.randn((B, H, T, d), generator=gen).cuda() for _ in range(2))
    pos = torch.randint(0, 100000, (B, T), generator=gen, dtype=torch.int32).cuda()

    def fwd(z):
        y = torch.empty_like(z)
        mita.mita_rope(p, z, None, y, None, pos=pos)
        return y.double()

    dx = torch.empty_like(x)
    mita.mita_rope_backward(p, g, None, dx, None, pos=pos)
    # the map is linear, so a difference over a step of 1 has no error but the roundings of its ends: each
    # element of y 8 2^-23 gain (|x0| + |x1|), of at most two that depend on a channel
    dots = (g.double() * fwd(x)).sum()
    size = 1.3 * (g.abs().double().sum() * 2 * x.abs().max().double())
    assert abs(float(dots - (dx.double() * x.double()).sum())) <= 16 * 2.0 ** -23 * float(size)
    for ch in (0, 1, rot // 2, rot - 1, rot, d - 1):
        if ch >= d:
            continue
        step = torch.zeros_like(x)
        step[..., ch] = 1.0
        diff = ((fwd(x + step) - fwd(x - step)) / 2 * g.double()).sum(-1)
        tol = 16 * 2.0 ** -23 * 1.3 * 2 * (float(x.abs().max()) + 1) * 2 * float(g.abs().max())
        assert float((diff - dx[..., ch].double()).abs().max()) <= tol


def test_streams_and_captured_calls():
    """A captured call reads its positions when it is replayed; a call on another stream waits for nothing."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    p = mita.RopeParams(4, 8, 2, 1, 128, 128)
    gen = torch.Generator().manual_seed(5)
    Q, K = (torch.randn((4, h, 1, 128), generator=gen).to(torch.bfloat16).cuda() for h in (8, 2))
    pos = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(x) for x in (Q, K)]
    mita.mita_rope(p, Q, K, *outs, pos=pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mita.mita_rope(p, Q, K, *outs, pos=pos)
        pos += 1
    side = torch.cuda.Stream()
    for step in range(3):
        want = [torch.empty_like(x) for x in (Q, K)]
        at = torch.full((4, 1), step, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        graph.replay()
        mita.mita_rope(p, Q, K, *want, pos=at, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
        assert int(pos[0, 0]) == step + 1


def test_rows_past_32_bits():
    """The last rows of tensors of more than 2^32 bytes, and strides that reach as far."""
    import torch
    import compressed_attention_adaptive_gb300 as mita
    B, H, T, d = 2, 17, 1 << 19, 128  # 2.3e9 elements of queries
    p = mita.RopeParams(B, H, 1, T, d, d)
    Q = torch.zeros((B, H, T, d), dtype=torch.bfloat16, device="cuda")
    K = torch.zeros((B, 1, T, d), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((3, d), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    Q[1, 16, -3:] = x
    K[1, 0, -3:] = x
    mita.mita_rope(p, Q, K, Q, K)
    at = np.arange(T - 3, T)
    freqs = mita.mita_rope_frequencies(d)
    _check("bf16", x, Q[1, 16, -3:], at, freqs, d, False, 1.0, False, "far rows")
    assert torch.equal(Q[1, 16, -3:], K[1, 0, -3:]) and not Q[0].any() and not Q[1, :16].any()
