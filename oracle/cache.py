"""fp64 restatement of the 4-bit cache format and of attention over cached rows.

Written from the definition in include/mita.h, with numpy only and nothing of
the CUDA library: ``quantise`` returns the values a block is held as (nearest
points of the two grids, ties to the even one), ``attention`` is softmax
attention of one head's rows over the keys that each row sees.
"""
import numpy as np

# magnitudes of the 4-bit codes (e2m1) and of the finite 8-bit scales (e4m3),
# ascending; the position's parity is that of the last bit
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(i % 8) * 2.0 ** -9 if i < 8 else (8 + i % 8) * 2.0 ** (i // 8 - 10) for i in range(127)])


def nearest(a, grid):
    """Nearest element of an ascending grid (a >= 0), ties to the even position,
    the last element beyond the grid."""
    a = np.minimum(np.asarray(a, np.float64), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, lo + lo % 2))
    return grid[pick]


def quantise(x, e=0):
    """Values (float64) that rows x [..., d] are held as with the exponents e
    (broadcast against x[..., 0])."""
    x = np.asarray(x, np.float64)
    e = np.broadcast_to(np.asarray(e), x.shape[:-1])[..., None, None]
    y = np.ldexp(x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16)), -e)
    a = np.abs(y).max(-1, keepdims=True)
    nan = np.isnan(a)
    s = nearest(np.where(nan, 0.0, a) / 6.0, E4M3)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, np.abs(y) / s, 0.0)
    v = np.copysign(nearest(np.where(np.isnan(q), 0.0, q), E2M1) * s, y)
    return np.ldexp(np.where(nan, np.nan, v), e).reshape(x.shape)


def attention(q, k, v, limits, scale):
    """q [rows, d], k and v [n, d] in fp64, limits [rows] = keys seen from the
    first on. Returns (o, lse, spread) with spread = sum_j w_j |v_j|, the
    magnitude that errors of the weights w act on."""
    o, spread = np.zeros((len(q), v.shape[1])), np.zeros((len(q), v.shape[1]))
    lse = np.full(len(q), -np.inf)
    for r, m in enumerate(limits):
        if m <= 0:
            continue
        z = (k[:m] @ q[r]) * scale
        p = np.exp(z - z.max())
        o[r], spread[r] = (p @ v[:m]) / p.sum(), (p @ np.abs(v[:m])) / p.sum()
        lse[r] = z.max() + np.log(p.sum())
    return o, lse, spread
