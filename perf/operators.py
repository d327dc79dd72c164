"""Cases and plain forms of the 4-bit key/value cache operators.

Three operators work on one paged cache: storing rows (``mita_cache_write``,
measured with the read-back that shows what it stored), reading rows back
(``mita_cache_read``) and attention of new rows over everything cached
(``mita_cache_attention``).

What the cache holds. A row of d channels is cut into blocks of 16. With e the
head's exponent (0 unless given) and a the block's largest |x * 2^-e|, the
block's scale is s = a / 6 rounded to e4m3 (4 significant bits, at most 448, at
least 2^-9 or zero) and each channel is x * 2^-e / s rounded to the nearest of
0, 1/2, 1, 3/2, 2, 3, 4, 6 with its sign (ties to the even code, beyond 6 to 6).
The value read back is code * s * 2^e; a block whose scale is zero reads zero.

Rows. A sequence b has len[b] cached tokens; a call's rows are its last
count[b] ones (T of them unless given), row t at position len - count + t, in
page table[b][position // page] at place position % page. Rows from count[b] on
are padding and stay as they were.

Attention. Row t of sequence b sees the keys j < len (causal: j <= its own
position), softmax(scale q.k) over them in each head, query heads in groups of
H / Hkv sharing a cache head; scale = 1 / sqrt(d).
"""
import math

import torch

own = False

_CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    bf, f4 = "bf16", "f32"
    mk = lambda name, op, B, H, Hkv, d, page, T, lo, hi, dtype, causal=False, exps=False: dict(
        name=name, op=op, B=B, H=H, Hkv=Hkv, d=d, page=page, T=T, lo=lo, hi=hi, dtype=dtype, causal=causal, exps=exps)
    return [
        # one new token of each of 48 running sequences, as every decoding step stores it
        mk("store_step", "store", 48, 8, 8, 128, 64, 1, 100, 5000, bf),
        # three padded prompts of a float32 model, 1000 rows at most, with per-head exponents
        mk("store_ragged_f32", "store", 3, 12, 12, 64, 16, 1000, 700, 1900, f4, exps=True),
        # the prompts of the long-context workload, whole
        mk("store_32k", "store", 2, 16, 16, 128, 64, 32768, 32768, 32768, bf),
        # the last 777 rows of five sequences, read for a second pass over them in float32
        mk("read_tail_f32", "read", 5, 4, 4, 128, 32, 777, 400, 3000, f4, exps=True),
        # both long prompts read back as the keys and values of a full forward pass
        mk("read_32k", "read", 2, 16, 16, 128, 64, 32768, 32768, 32768, bf),
        # a single short conversation, one token: latency counts
        mk("decode_short", "attend", 1, 16, 16, 128, 64, 1, 1000, 1000, bf),
        # one token after each prompt of the long-context workload, a cache head for every query head
        mk("decode_32k", "attend", 2, 16, 16, 128, 64, 1, 32768, 32768, bf),
        # one token of a very long context, eight query heads to a cache head
        mk("decode_131k_grouped", "attend", 1, 64, 8, 128, 128, 1, 131072, 131072, bf),
        # a serving batch of very unlike lengths, small pages
        mk("decode_batch", "attend", 64, 32, 8, 128, 16, 1, 33, 8191, bf, exps=True),
        # five drafted tokens checked at once, an odd group, narrow heads
        mk("draft_narrow", "attend", 9, 24, 8, 64, 32, 5, 501, 20011, bf, causal=True),
        # eight drafted tokens of a grouped model: 64 query rows a cache head
        mk("draft_grouped", "attend", 4, 64, 8, 128, 64, 8, 9000, 16384, bf, causal=True),
        # float32 rows over the vision workload's 128 x 128 tokens
        mk("decode_f32", "attend", 8, 12, 12, 64, 64, 1, 16384, 16384, f4, exps=True),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["store", "read", "attend", "attend"])
    c = dict(op=op, d=rng.choice([64, 128]), page=rng.choice([16, 32, 48, 64, 128]),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), exps=rng.random() < 0.4)
    c["Hkv"] = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    if op == "attend":
        c["H"] = c["Hkv"] * rng.choice([1, 1, 2, 3, 4, 5, 8])
        c["T"] = rng.choice([1, 1, 1, 2, 3, 4, 6, 8])
        c["causal"] = rng.random() < 0.7
        c["B"] = logint(1, 64)
        tokens = logint(c["B"] * 64, 500000 // c["Hkv"] if c["H"] * c["T"] <= 64 else 100000 // c["Hkv"])
        c["hi"] = max(8, min(131072, tokens // c["B"]))
        c["lo"] = rng.choice([c["hi"], max(1, c["hi"] // 3), max(1, c["hi"] // 40)])
    else:
        c["H"], c["causal"] = c["Hkv"], False
        c["B"] = logint(1, 64)
        c["T"] = min(32768, max(1, logint(c["B"], 500000 // c["Hkv"]) // c["B"]))
        c["hi"] = c["T"] + rng.choice([0, 1, logint(2, 4000)])
        c["lo"] = rng.choice([c["hi"], max(1, c["hi"] // 2)])
    return c


def _lens(case):
    """Cached tokens of each sequence, spread over [lo, hi] with both ends in."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if lo == hi or B == 1:
        return [hi] * B
    return [hi, lo] + [lo + int((hi - lo) * ((b * 0.6180339887) % 1.0)) for b in range(2, B)]


def _counts(case):
    return [min(case["T"], n) for n in _lens(case)]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _inputs(case, seed):
    """Inputs from the seed alone: what both sides and the definition start from."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 17)
    B, H, Hkv, d, page, T = (case[x] for x in ("B", "H", "Hkv", "d", "page", "T"))
    dt = _dtype(case)
    lens, counts = _lens(case), _counts(case)
    cols = max(-(-n // page) for n in lens)
    n_pages = sum(-(-n // page) for n in lens) + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((B, cols), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = perm[at:at + k]
        at += k
    x = dict(table=table, n_pages=n_pages, cols=cols, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             counts=torch.tensor(counts, dtype=torch.int32, device=dev), exps=None)
    if case["exps"]:
        x["exps"] = torch.randint(-4, 3, (2, Hkv), generator=g, device=dev, dtype=torch.int32)
    rows = T if case["op"] == "store" else max(lens)
    # keys with a few strong channels and an offset, values small, as a model's projections give them
    cs = torch.exp(0.4 * torch.randn((Hkv, 1, d), generator=g, device=dev))
    off = 0.5 * torch.randn((Hkv, 1, d), generator=g, device=dev)

    def rows_of(make, e):
        out = torch.empty((B, Hkv, rows, d), dtype=dt, device=dev)
        up = 1.0 if e is None else torch.exp2(e.float()).view(Hkv, 1, 1)
        for b in range(B):
            out[b] = (make(torch.randn((Hkv, rows, d), generator=g, device=dev)) * up).to(dt)
        return out

    ex = x["exps"]
    x["K"] = rows_of(lambda r: r * cs + off, None if ex is None else ex[0])
    x["V"] = rows_of(lambda r: 0.6 * r, None if ex is None else ex[1])
    if case["op"] == "attend":
        x["Q"] = torch.randn((B, H, T, d), generator=g, device=dev).to(dt)
    return x


# ---------------------------------------------------------------- plain form


def _quantise(x, e):
    """Codes (0..15, bit 3 the sign) and scales of rows [..., d] in 32 bits; every
    step is exact but the two roundings the format defines."""
    y = x.float()
    if e is not None:
        y = torch.ldexp(y, -e)
    y = y.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    raw = y.abs().amax(-1) / 6.0
    m, p = torch.frexp(raw)
    step = torch.ldexp(torch.ones_like(raw), torch.clamp(p - 1, min=-6) - 3)
    s = torch.clamp(torch.round(raw / step) * step, max=448.0)
    q = torch.where(s[..., None] > 0, y.abs() / torch.where(s > 0, s, torch.ones_like(s))[..., None],
                    torch.zeros_like(y))
    code = torch.zeros_like(q, dtype=torch.uint8)
    for t, open_ in ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)):
        code += (q > t if open_ else q >= t).to(torch.uint8)
    code |= (y < 0).to(torch.uint8) << 3
    return code.reshape(x.shape), s.to(torch.float16)


def _values(code, s, e):
    grid = torch.tensor(_CODES + tuple(-c for c in _CODES), device=code.device)
    v = grid[code.long()].reshape(code.shape[:-1] + (code.shape[-1] // 16, 16)) * s.float()[..., None]
    v = v.reshape(code.shape)
    return v if e is None else torch.ldexp(v, e)


def _pool(x, case):
    """Plain cache: packed codes and scales per page, head and place."""
    n, Hkv, page, d = x["n_pages"], case["Hkv"], case["page"], case["d"]
    dev = x["table"].device
    return [(torch.zeros((n, Hkv, page, d // 2), dtype=torch.uint8, device=dev),
             torch.zeros((n, Hkv, page, d // 16), dtype=torch.float16, device=dev)) for _ in range(2)]


def _plan(x, case, lens, counts):
    """Where the call's rows are: sequence, row, page and place of each."""
    bi = torch.tensor([b for b, c in enumerate(counts) for _ in range(c)], device=x["table"].device)
    ti = torch.cat([torch.arange(c) for c in counts]).to(bi.device)
    first = torch.tensor([n - c for n, c in zip(lens, counts)], device=bi.device)
    pos = first[bi] + ti
    return bi, ti, x["table"][bi, pos // case["page"]].long(), pos % case["page"]


def _plain_store(x, pool, plan, K, V):
    bi, ti, pg, at = plan
    for i, X in enumerate((K, V)):
        code, s = _quantise(X[bi, :, ti], None if x["exps"] is None else x["exps"][i].view(1, -1, 1))
        pool[i][0][pg, :, at] = code[..., 0::2] | (code[..., 1::2] << 4)
        pool[i][1][pg, :, at] = s


def _plain_rows(x, pool, case, pg, at, i):
    """Values [rows, Hkv, d] of the rows at places `at` of pages `pg` in 32 bits."""
    packed = pool[i][0][pg, :, at]
    code = torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[:-1] + (case["d"],))
    return _values(code, pool[i][1][pg, :, at], None if x["exps"] is None else x["exps"][i].view(1, -1, 1))


def _plain_read(x, pool, case, plan):
    bi, ti, pg, at = plan
    outs = []
    for i in range(2):
        out = torch.zeros((case["B"], case["Hkv"], case["T"], case["d"]), dtype=_dtype(case),
                          device=x["table"].device)
        out[bi, :, ti] = _plain_rows(x, pool, case, pg, at, i).to(out.dtype)
        outs.append(out)
    return tuple(outs)


def _plain_attend(x, pool, case, lens, counts):
    B, H, Hkv, T, d = (case[k] for k in ("B", "H", "Hkv", "T", "d"))
    out = torch.zeros((B, H, T, d), dtype=_dtype(case), device=x["table"].device)
    for b in range(B):
        n, c = lens[b], counts[b]
        pos = torch.arange(n, device=out.device)
        pg, at = x["table"][b, pos // case["page"]].long(), pos % case["page"]
        k, v = (_plain_rows(x, pool, case, pg, at, i).transpose(0, 1) for i in range(2))
        q = x["Q"][b, :, :c].float().reshape(Hkv, (H // Hkv) * c, d)
        s = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
        if case["causal"]:
            last = pos[n - c:].repeat(H // Hkv)
            s = torch.where(pos[None, :] <= last[:, None], s,
                            torch.full_like(s, -math.inf))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        out[b, :, :c] = o.reshape(H, c, d).to(out.dtype)
    return out


# ------------------------------------------------------------ what is measured


def prepare(case, seed):
    x = _inputs(case, seed)
    lens, counts = _lens(case), _counts(case)
    st = dict(case=case, x=x, lens=lens, counts=counts)
    K, V = x["K"], x["V"]
    if own:
        import compressed_attention_adaptive_gb300 as mita
        dt = {"bf16": mita.BF16, "f32": mita.F32}[case["dtype"]]
        flags = mita.FLAG_CAUSAL if case["causal"] else 0
        p = mita.CacheParams(case["B"], case["H"], case["Hkv"], case["T"], case["d"], case["page"], x["n_pages"],
                             x["cols"], flags=flags, dtype=dt)
        st["p"] = p
        st["cache"] = torch.zeros(mita.mita_cache_size(p), dtype=torch.uint8, device="cuda")
        st["ws"] = mita.cache_workspace(p)
        if case["op"] != "store":  # a cache filled by the prompts before
            fill = mita.CacheParams(case["B"], case["Hkv"], case["Hkv"], K.shape[2], case["d"], case["page"],
                                    x["n_pages"], x["cols"], dtype=dt)
            ws = mita.cache_workspace(fill)
            mita.mita_cache_write(fill, K, V, st["cache"], x["table"], x["lens"], ws, counts=x["lens"],
                                  exps=x["exps"])
            mita.mita_device_status(ws)
        if case["op"] == "attend":
            st["O"] = torch.zeros_like(x["Q"])
        else:
            shape = (case["B"], case["Hkv"], case["T"], case["d"])
            st["Kr"], st["Vr"] = (torch.zeros(shape, dtype=_dtype(case), device="cuda") for _ in range(2))
    else:
        st["pool"] = _pool(x, case)
        if case["op"] != "store":
            _plain_store(x, st["pool"], _plan(x, case, lens, lens), K, V)
        st["plan"] = _plan(x, case, lens, counts)
    if case["op"] != "store":
        del x["K"], x["V"], K, V
    return st


def run(st):
    case, x = st["case"], st["x"]
    op = case["op"]
    if own:
        import compressed_attention_adaptive_gb300 as mita
        p = st["p"]
        if op == "attend":
            mita.mita_cache_attention(p, x["Q"], st["cache"], x["table"], x["lens"], st["O"], st["ws"],
                                      counts=x["counts"], exps=x["exps"])
            return st["O"]
        if op == "store":
            mita.mita_cache_write(p, x["K"], x["V"], st["cache"], x["table"], x["lens"], st["ws"],
                                  counts=x["counts"], exps=x["exps"])
        mita.mita_cache_read(p, st["cache"], x["table"], x["lens"], st["Kr"], st["Vr"], st["ws"],
                             counts=x["counts"], exps=x["exps"])
        return st["Kr"], st["Vr"]
    if op == "attend":
        return _plain_attend(x, st["pool"], case, st["lens"], st["counts"])
    if op == "store":
        _plain_store(x, st["pool"], st["plan"], x["K"], x["V"])
    return _plain_read(x, st["pool"], case, st["plan"])


def work(case):
    B, H, Hkv, T, d = (case[k] for k in ("B", "H", "Hkv", "T", "d"))
    lens, counts = _lens(case), _counts(case)
    elem = 2 if case["dtype"] == "bf16" else 4
    token = 2 * Hkv * (d // 2 + d // 16)  # one token's keys and values in the cache
    ints = 4 * (2 * B + sum(-(-n // case["page"]) for n in lens))
    rows = sum(counts)
    if case["op"] == "attend":
        seen = sum(sum(n - (c - 1 - t) if case["causal"] else n for t in range(c)) for n, c in zip(lens, counts))
        return {"bytes": sum(lens) * token + 2 * rows * H * d * elem + ints, "flops": 4 * H * d * seen}
    plain = 2 * rows * Hkv * d * elem  # keys and values as the caller holds them
    if case["op"] == "store":  # read the rows, write the cache; read the cache, write the rows
        return {"bytes": 2 * (plain + rows * token) + ints, "flops": 2 * 4 * rows * Hkv * d}
    return {"bytes": plain + rows * token + ints, "flops": 2 * rows * Hkv * d}


# ------------------------------------------- the definition in 64 bits, by itself


def _def_values(x, e):
    """Values in 64 bits that rows x (64 bits) are held as, straight from the
    format: nearest points on the two grids, ties to the even one."""
    y = x * torch.exp2(-e) if e is not None else x
    y = y.reshape(x.shape[:-1] + (-1, 16))
    a = y.abs().amax(-1, keepdim=True) / 6.0
    # the 127 finite e4m3 magnitudes; even positions have an even last bit
    mags = torch.tensor([(i % 8) * 2.0 ** -9 if i < 8 else (8 + i % 8) * 2.0 ** (i // 8 - 10) for i in range(127)],
                        dtype=torch.float64, device=x.device)
    s = _nearest(a, mags)
    grid = torch.tensor(_CODES, dtype=torch.float64, device=x.device)
    r = torch.where(s > 0, y.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    v = torch.copysign(_nearest(r, grid) * s, y).reshape(x.shape)
    return v * torch.exp2(e) if e is not None else v


def _nearest(a, grid):
    """Nearest element of an ascending grid, ties to the even position."""
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    pick = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))
    return grid[pick]


def exact(case, seed):
    x = _inputs(case, seed)
    lens, counts = _lens(case), _counts(case)
    e = [None if x["exps"] is None else x["exps"][i].double().view(-1, 1, 1) for i in range(2)]
    B, H, Hkv, T, d = (case[k] for k in ("B", "H", "Hkv", "T", "d"))
    if case["op"] != "attend":
        outs = []
        for i, X in enumerate((x["K"], x["V"])):
            out = torch.zeros((B, Hkv, T, d), dtype=torch.float64, device=X.device)
            for b in range(B):
                c = counts[b]
                src = X[b, :, :c] if case["op"] == "store" else X[b, :, lens[b] - c:lens[b]]
                for h in range(Hkv):
                    out[b, h, :c] = _def_values(src[h:h + 1].double(), None if e[i] is None else e[i][h:h + 1])[0]
            outs.append(out)
        return tuple(outs)
    out = torch.zeros((B, H, T, d), dtype=torch.float64, device=x["Q"].device)
    G = H // Hkv
    for b in range(B):
        n, c = lens[b], counts[b]
        for h in range(Hkv):
            k, v = (_def_values(X[b, h:h + 1, :n].double(), None if e[i] is None else e[i][h:h + 1])[0]
                    for i, X in enumerate((x["K"], x["V"])))
            for t in range(c):
                m = n - (c - 1 - t) if case["causal"] else n
                z = x["Q"][b, h * G:(h + 1) * G, t].double() @ k[:m].T / math.sqrt(d)
                w = torch.exp(z - z.amax(-1, keepdim=True))
                out[b, h * G:(h + 1) * G, t] = (w @ v[:m]) / w.sum(-1, keepdim=True)
    return out
