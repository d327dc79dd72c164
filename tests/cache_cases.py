"""Shared by the tests of the 4-bit cache: a pool with its page table, and the
bounds that outputs are held to."""
import numpy as np

from oracle import cache as ocache


class Pool:
    """A pool on the GPU, its table (pages in random order) and the values that
    the oracle says it holds: rows[b] = (K, V), each [H_kv, len, d] in fp64."""

    def __init__(self, lens, Hkv, d, page, dtype, seed=0, exps=None, H=None, T=1, flags=0, scale=0.0, cols=None,
                 fill=0xff, make=None):
        import torch
        import compressed_attention_adaptive_gb300 as mita
        self.mita, self.torch = mita, torch
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.d, self.page, self.dtype = list(lens), Hkv, d, page, dtype
        B, H = len(lens), H or Hkv
        need = [-(-n // page) for n in lens]
        self.cols = cols or max(1, max(need))
        self.n_pages = sum(need) + 2
        perm = rng.permutation(self.n_pages).astype(np.int32)
        table = np.full((B, self.cols), 2 ** 31 - 1, np.int32)  # entries past a sequence's end are not read
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = perm[at:at + k]
            at += k
        self.table = torch.from_numpy(table).cuda()
        self.len_t = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.exps_np = None if exps is None else np.asarray(exps, np.int32)
        self.exps = None if exps is None else torch.from_numpy(self.exps_np).cuda()
        self.p = mita.CacheParams(B, H, Hkv, T, d, page, self.n_pages, self.cols, scale, flags,
                                  mita.BF16 if dtype == "bf16" else mita.F32)
        self.cache = torch.full((mita.mita_cache_size(self.p),), fill, dtype=torch.uint8, device="cuda")
        self.ws = mita.cache_workspace(self.p)
        self.ws.fill_(0xff)  # nothing of a call may rest on what the workspace held
        longest = max(1, max(lens))
        K, V = (make or self.rows)(rng, (B, Hkv, longest, d))
        self.K, self.V = (torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(self.td).cuda() for x in (K, V))
        self.fill_p = mita.CacheParams(B, Hkv, Hkv, longest, d, page, self.n_pages, self.cols, 0.0, 0, self.p.dtype)
        self.fill_ws = mita.cache_workspace(self.fill_p)
        if max(lens) > 0:
            mita.mita_cache_write(self.fill_p, self.K, self.V, self.cache, self.table, self.len_t, self.fill_ws,
                                  counts=self.len_t, exps=self.exps)
            mita.mita_device_status(self.fill_ws)

    @property
    def td(self):
        return self.torch.bfloat16 if self.dtype == "bf16" else self.torch.float32

    @staticmethod
    def rows(rng, shape):
        """Keys with strong channels and an offset, smaller values."""
        d = shape[-1]
        return (rng.standard_normal(shape) * np.exp(0.5 * rng.standard_normal(d)) + 0.5 * rng.standard_normal(d),
                0.7 * rng.standard_normal(shape))

    def held(self, b, which, n=None):
        """[H_kv, len, d] fp64: what the oracle says sequence b holds."""
        x = (self.K, self.V)[which][b, :, :self.lens[b] if n is None else n].float().cpu().numpy()
        e = 0 if self.exps_np is None else self.exps_np[which][:, None]
        return ocache.quantise(x, e)


def attention_bound(dtype, tensor_cores, o, spread, q, k, v, limits, scale):
    """Allowed |gpu - oracle| per element of a head's rows, counted from the
    roundings (u = half a step: bf16 2^-8, half 2^-11, float 2^-24):
      - the output's own rounding, u |o|;
      - a score z is a sum of d products in fp32 and one product by the scale:
        off by at most (d + 4) 2^-23 of scale sum |q_c k_c| (2^-23, not 2^-24,
        for sums that cut instead of rounding), and exp of it is off by that
        much relative, the weights' sum likewise; the difference z - max and the
        exponential itself: 2^-21 (1 + |z - max|), with |z - max| at most twice
        the magnitude above and at most 64 where the weight is not nothing;
      - bf16 on tensor cores rounds the weights to halves: 2^-11 each, or 2^-25 of
        the largest below 2^-14 of it, against a sum of at least the largest;
        float32 makes two halves of a query's entry and of a weight: 2^-23 each,
        which the next two lines' chains and the scores' d additions have room for;
      - sums over keys in fp32: 2^-23 for every addition in a chain, of which
        there are at most one per 16 keys and 64 more for the joins."""
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    out = np.zeros_like(o)
    for r, m in enumerate(limits):
        if m <= 0:
            continue
        mag = scale * (np.abs(k[:m]) @ np.abs(q[r])).max()
        rel = 2 * (k.shape[1] + 4) * 2.0 ** -23 * mag + 2.0 ** -21 * (1 + min(64.0, 2 * mag))
        rel += (m / 16 + 64) * 2.0 ** -23
        if tensor_cores:
            rel += 2.0 ** -11
        out[r] = u * np.abs(o[r]) + rel * spread[r]
        if tensor_cores:
            out[r] += 2.0 ** -25 * np.abs(v[:m]).sum(0)
    return out * (1 + 2.0 ** -6) + 1e-30  # products of two of these errors
