"""Cases and plain forms of the operators for long generation: rotary positions,
the attention weight that cached tokens receive, and eviction by it.

Rotation (``mita_rope``, ``mita_rope_backward``). Of a row's first ``rot``
channels pair i is (i, i + rot/2), or (2i, 2i + 1) interleaved; at position p it
is turned by the angle p * freq[i] and scaled by a gain, the other channels are
copied. The backward pass is the transposed map. Queries and keys go through one
call, from any strides (a projection's [B, T, heads, d], say) into [B, heads, T, d].

Weights (``mita_cache_weights``). acc[b, h, j] of cached token j and cache head h
becomes decay * acc (0 for the call's own tokens) plus the sum, over the call's
rows and the query heads of h that see j, of exp(scale q.k_j - lse), lse being
the row's log sum from the attention.

Eviction (``mita_cache_evict``). A sequence with more than keep[b] tokens keeps
that many: the first ``first``, the last ``recent``, and of the others those with
the largest acc (ties to the lower place), each cache head its own. Kept rows at
or behind the new length move, in order, into the places freed before it. It is
measured with the read-back of what is kept. src[b, h, j] is the place that the
row now at j had.

The cache's format: a row of d channels is cut into blocks of 16; with e the
head's exponent (0 unless given) and a the block's largest |x * 2^-e|, s = a / 6
rounded to e4m3, and each channel is x * 2^-e / s rounded to the nearest of 0, 1/2,
1, 3/2, 2, 3, 4, 6 with its sign, ties to the even code. Position i of sequence b
is place i % page of page table[b][i // page].
"""
import math

import torch

own = False

_CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    bf, f4 = "bf16", "f32"

    def rope(name, op, B, H, Hkv, T, d, rot, layout, source, dtype, far, scaling="none", factor=1.0):
        return dict(name=name, op=op, B=B, H=H, Hkv=Hkv, T=T, d=d, rot=rot, layout=layout, source=source, dtype=dtype,
                    far=far, scaling=scaling, factor=factor)

    def weigh(name, B, H, Hkv, d, page, T, lo, hi, dtype, causal=False, exps=False, decay=1.0):
        return dict(name=name, op="weigh", B=B, H=H, Hkv=Hkv, d=d, page=page, T=T, lo=lo, hi=hi, dtype=dtype,
                    causal=causal, exps=exps, decay=decay)

    def evict(name, B, Hkv, d, page, lo, hi, keep, first, recent, dtype):
        return dict(name=name, op="evict", B=B, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi, keep=keep, first=first,
                    recent=recent, dtype=dtype)

    return [
        # one new token of each of 64 running sequences at far positions of a scaled context: latency counts
        rope("rope_step", "rope", 64, 32, 8, 1, 128, 128, "half", "proj", bf, 131072, "parts", 8.0),
        # the prompts of the long-context workload, from the projection's order into the heads'
        rope("rope_32k", "rope", 2, 16, 16, 32768, 128, 128, "half", "proj", bf, 0),
        # three short prompts of a float32 model, part of an odd head in the interleaved order
        rope("rope_part_f32", "rope", 3, 12, 12, 1000, 80, 20, "interleaved", "heads", f4, 5000, "linear", 4.0),
        # gradients of a grouped model's rotated queries and keys, as a training step has them
        rope("rope_back_131k", "rope_back", 1, 8, 2, 131072, 128, 64, "interleaved", "heads", bf, 0, "ntk", 2.0),
        # a single short conversation, one token: latency counts
        weigh("weigh_short", 1, 16, 16, 128, 64, 1, 1000, 1000, bf),
        # one token after each prompt of the long-context workload
        weigh("weigh_32k", 2, 16, 16, 128, 64, 1, 32768, 32768, bf),
        # a serving batch of very unlike lengths, small pages, sums that fade
        weigh("weigh_batch", 64, 32, 8, 128, 16, 1, 33, 8191, bf, exps=True, decay=0.95),
        # drafted tokens of a float32 model with narrow heads and an odd group
        weigh("weigh_drafts_f32", 9, 24, 8, 64, 32, 5, 501, 20011, f4, causal=True),
        # a prompt's last 32 tokens, eight query heads to a cache head, decide what is kept of it
        weigh("weigh_window", 2, 64, 8, 128, 64, 32, 30001, 32768, bf, causal=True, decay=0.0),
        # running sequences that went 64 tokens past their budget
        evict("evict_step", 16, 8, 128, 64, 2112, 2112, 2048, 4, 256, bf),
        # a ragged batch: some sequences within their budget, others far over it
        evict("evict_batch", 24, 6, 64, 48, 700, 9001, 1500, 0, 33, f4),
        # both long prompts cut to an eighth
        evict("evict_32k", 2, 16, 128, 64, 32768, 32768, 4096, 16, 512, bf),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["rope", "rope_back", "weigh", "weigh", "evict", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    if op.startswith("rope"):
        d = rng.choice([40, 64, 72, 80, 96, 128, 160, 256])
        c = dict(op=op, B=logint(1, 64), Hkv=Hkv, H=Hkv * rng.choice([1, 1, 2, 3, 4, 8]), d=d,
                 rot=rng.choice([d, d, d // 2, d // 4]), layout=rng.choice(["half", "interleaved"]),
                 source=rng.choice(["proj", "heads"]), dtype=dtype, far=rng.choice([0, logint(10, 1000000)]),
                 scaling=rng.choice(["none", "linear", "ntk", "parts"]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]))
        rows = logint(1, 60000000 // ((c["H"] + Hkv) * d * c["B"])) if rng.random() < 0.8 else 1
        c["T"] = max(1, rows)
        return c
    c = dict(op=op, Hkv=Hkv, d=rng.choice([64, 128]), page=rng.choice([16, 32, 48, 64, 128]), dtype=dtype)
    if op == "weigh":
        c["H"] = Hkv * rng.choice([1, 1, 2, 3, 4, 5, 8])
        c["T"] = rng.choice([1, 1, 1, 2, 3, 5, 8, 16, 33, 64])
        c["causal"], c["exps"] = rng.random() < 0.7, rng.random() < 0.4
        c["decay"] = rng.choice([0.0, 0.9, 1.0])
        c["B"] = logint(1, 64)
        most = min(1000000 // Hkv, 130000000 // (c["H"] * c["T"]))
        c["hi"] = max(8, min(131072, logint(c["B"] * 64, most) // c["B"]))
    else:
        c["B"] = logint(1, 64)
        c["hi"] = max(8, min(131072, logint(c["B"] * 64, 1000000 // Hkv) // c["B"]))
        c["first"], c["recent"] = rng.choice([0, 1, 4, 16]), rng.choice([0, 1, 32, logint(1, max(1, c["hi"] // 4))])
        c["keep"] = max(1, c["first"] + c["recent"], int(c["hi"] * rng.choice([0.05, 0.3, 0.9, 0.99])))
    c["lo"] = rng.choice([c["hi"], max(1, c["hi"] // 3), max(1, c["hi"] // 40)])
    return c


def _lens(case):
    """Cached tokens of each sequence, spread over [lo, hi] with both ends in."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if lo == hi or B == 1:
        return [hi] * B
    return [hi, lo] + [lo + int((hi - lo) * ((b * 0.6180339887) % 1.0)) for b in range(2, B)]


def _counts(case):
    return [min(case["T"], n) for n in _lens(case)]


def _keeps(case):
    """Budgets of the sequences: keep, a little less for every third one."""
    least = max(1, case["first"] + case["recent"])
    return [max(least, case["keep"] - (case["keep"] // 7 if b % 3 == 2 else 0)) for b in range(case["B"])]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ------------------------------------------------------------------- inputs


def _freqs(case):
    """Radians per position of the pairs, in Python's own floats."""
    rot, factor, base = case["rot"], case["factor"], 10000.0
    if case["scaling"] == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    if case["scaling"] == "parts":  # 8192 positions at first; below 1 turn over them scaled, from 4 on not
        part = [min(1.0, max(0.0, (8192.0 * x / (2.0 * math.pi) - 1.0) / 3.0)) for x in f]
        f = [x * (g + (1.0 - g) / factor) for x, g in zip(f, part)]
    return f


def _gain(case):
    return 1.0 + 0.1 * math.log(case["factor"]) if case["scaling"] == "parts" else 1.0


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    return g


def _rope_inputs(case, seed):
    """Rows as they lie in the caller's buffers, seen as [B, heads, T, d], and positions."""
    g = _generator(seed)
    B, H, Hkv, T, d = (case[k] for k in ("B", "H", "Hkv", "T", "d"))
    if case["source"] == "proj":  # one product's output: queries, keys and values of a token in a row
        both = torch.randn((B, T, H + 2 * Hkv, d), generator=g, device="cuda", dtype=_dtype(case)).transpose(1, 2)
        Q, K = both[:, :H], both[:, H:H + Hkv]
    else:
        Q, K = (torch.randn((B, h, T, d), generator=g, device="cuda", dtype=_dtype(case)) for h in (H, Hkv))
    at = torch.arange(T, device="cuda", dtype=torch.int32).expand(B, T)
    if case["far"]:
        at = at + torch.randint(0, case["far"], (B, 1), generator=g, device="cuda", dtype=torch.int32)
    return Q, K, at.contiguous()


def _cache_inputs(case, seed):
    g = _generator(seed)
    dev = torch.device("cuda")
    B, Hkv, d, page = (case[k] for k in ("B", "Hkv", "d", "page"))
    lens = _lens(case)
    need = [-(-n // page) for n in lens]
    cols, n_pages = max(need), sum(need) + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((B, cols), dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    x = dict(table=table, n_pages=n_pages, cols=cols, lens=torch.tensor(lens, dtype=torch.int32, device=dev), exps=None)
    if case.get("exps"):
        x["exps"] = torch.randint(-4, 3, (2, Hkv), generator=g, device=dev, dtype=torch.int32)
    # keys with a few strong channels and an offset, values small, as a model's projections give them
    cs = torch.exp(0.4 * torch.randn((Hkv, 1, d), generator=g, device=dev))
    off = 0.5 * torch.randn((Hkv, 1, d), generator=g, device=dev)
    up = [1.0, 1.0] if x["exps"] is None else [torch.exp2(e.float()).view(Hkv, 1, 1) for e in x["exps"]]
    shape = (B, Hkv, max(lens), d)
    x["K"] = ((torch.randn(shape, generator=g, device=dev) * cs + off) * up[0]).to(_dtype(case))
    x["V"] = (0.6 * torch.randn(shape, generator=g, device=dev) * up[1]).to(_dtype(case))
    # sums of weights fall off over several powers of ten; some tokens have had none
    wide = (B, Hkv, cols * page)
    acc = torch.exp(2.0 * torch.randn(wide, generator=g, device=dev) - 4.0)
    x["acc"] = torch.where(torch.rand(wide, generator=g, device=dev) < 0.02, torch.zeros_like(acc), acc)
    if case["op"] == "weigh":  # of a few dozen rows, not of many: what the call adds counts
        x["acc"] *= 50.0 / max(lens)
    else:
        x["keep"] = torch.tensor(_keeps(case), dtype=torch.int32, device=dev)
        return x
    H, T = case["H"], case["T"]
    x["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=dev)
    x["Q"] = torch.randn((B, H, T, d), generator=g, device=dev).to(_dtype(case))
    # the rows' log sums, as the attention before this call returned them
    s = _scores(case, x, _held(x["K"], None if x["exps"] is None else x["exps"][0].view(1, -1, 1, 1)))
    x["lse"] = torch.logsumexp(s, -1).reshape(B, H, T)
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
    code = ((q > 0.25).to(torch.uint8) + (q >= 0.75).to(torch.uint8) + (q > 1.25).to(torch.uint8)
            + (q >= 1.75).to(torch.uint8) + (q > 2.5).to(torch.uint8) + (q >= 3.5).to(torch.uint8)
            + (q > 5.0).to(torch.uint8))
    code |= (y < 0).to(torch.uint8) << 3
    return code.reshape(x.shape), s.to(torch.float16)


def _values(code, s, e):
    grid = torch.tensor(_CODES + tuple(-c for c in _CODES), device=code.device)
    v = grid[code.long()].reshape(code.shape[:-1] + (code.shape[-1] // 16, 16)) * s.float()[..., None]
    v = v.reshape(code.shape)
    return v if e is None else torch.ldexp(v, e)


def _held(x, e):
    return _values(*_quantise(x, e), e)


def _fill(x, case, X, e):
    """Plain cache of rows X [B, Hkv, n, d]: packed codes and scales per page, head and place."""
    n, Hkv, page, d = x["n_pages"], case["Hkv"], case["page"], case["d"]
    codes = torch.zeros((n, Hkv, page, d // 2), dtype=torch.uint8, device=X.device)
    scales = torch.zeros((n, Hkv, page, d // 16), dtype=torch.float16, device=X.device)
    j = torch.arange(X.shape[2], device=X.device)
    b, j = torch.nonzero(j < x["lens"][:, None], as_tuple=True)
    code, s = _quantise(X[b, :, j], None if e is None else e.view(1, -1, 1))
    at = x["table"][b, j // page].long()
    codes[at, :, j % page] = code[..., 0::2] | (code[..., 1::2] << 4)
    scales[at, :, j % page] = s
    return codes, scales


def _rows(x, case, pool, e, n):
    """Values [B, Hkv, n, d] of the first n places of the sequences in 32 bits (whatever is there behind their ends)."""
    j = torch.arange(n, device=pool[0].device)
    at = x["table"][:, j // case["page"]].long()
    packed, s = (t[at, :, (j % case["page"]).expand_as(at)].transpose(1, 2) for t in pool)
    code = torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[:-1] + (case["d"],))
    return _values(code, s, None if e is None else e.view(1, -1, 1, 1))


def _scores(case, x, k):
    """scale q.k [B, Hkv, G * T, n], -infinity where a row does not see the key or is padding."""
    B, H, Hkv, T, d = (case[c] for c in ("B", "H", "Hkv", "T", "d"))
    s = torch.matmul(x["Q"].float().reshape(B, Hkv, (H // Hkv) * T, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    j = torch.arange(k.shape[2], device=k.device)
    t = torch.arange(T, device=k.device)
    end = x["lens"][:, None].expand(B, T)
    if case["causal"]:
        end = end - x["counts"][:, None] + t + 1
    end = torch.where(t < x["counts"][:, None], end, torch.zeros_like(end))
    seen = (j < end[..., None]).repeat(1, H // Hkv, 1)
    return s.masked_fill_(~seen[:, None], -math.inf)


def _plain_weigh(st):
    case, x = st["case"], st["x"]
    n = max(_lens(case))
    s = _scores(case, x, _rows(x, case, st["pool"][0], None if x["exps"] is None else x["exps"][0], n))
    lse = x["lse"].reshape(s.shape[:-1])[..., None]
    w = torch.where(s == -math.inf, torch.zeros_like(s), torch.exp(s - lse)).sum(2)
    j = torch.arange(n, device=w.device)
    old = (j < (x["lens"] - x["counts"])[:, None])[:, None]
    if case["decay"]:
        w = w + torch.where(old, case["decay"] * x["acc"][..., :n], torch.zeros_like(w))
    out = torch.zeros_like(x["acc"])
    out[..., :n] = torch.where((j < x["lens"][:, None])[:, None], w, torch.zeros_like(w))
    return out


def _plain_evict(st):
    case, x = st["case"], st["x"]
    page, acc = case["page"], x["acc"]
    n, now = max(_lens(case)), torch.minimum(x["lens"], x["keep"])
    j = torch.arange(n, device=acc.device)
    len_, new = x["lens"].view(-1, 1, 1), now.view(-1, 1, 1)
    always = (j < case["first"]) | (j >= len_ - case["recent"])
    rank = torch.where(j < len_, torch.where(always, torch.full_like(acc[..., :n], math.inf), acc[..., :n]),
                       torch.full_like(acc[..., :n], -1.0))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(rank, dtype=torch.bool).scatter_(-1, order, (j < new).expand_as(order))
    b, h, to = torch.nonzero(~kept & (j < new), as_tuple=True)
    _, _, frm = torch.nonzero(kept & (j >= new), as_tuple=True)
    src = torch.where((j < new).expand_as(rank), j, torch.zeros_like(j)).to(torch.int32)
    src[b, h, to] = frm.to(torch.int32)
    at, into = (x["table"][b, i // page].long() for i in (frm, to))
    (kc, ks), (vc, vs) = st["pool"]
    kc[into, h, to % page], ks[into, h, to % page] = kc[at, h, frm % page], ks[at, h, frm % page]
    vc[into, h, to % page], vs[into, h, to % page] = vc[at, h, frm % page], vs[at, h, frm % page]
    most = max(_keeps(case))
    live = (torch.arange(min(n, most), device=acc.device) < new)[..., None]
    K, V = (torch.where(live, _rows(x, case, p, None, live.shape[2]), torch.zeros((), device=acc.device)).to(_dtype(case))
            for p in st["pool"])
    sums, place = torch.zeros_like(acc), torch.zeros(acc.shape, dtype=torch.int32, device=acc.device)
    sums[..., :n] = torch.where(j < new, torch.gather(acc, -1, src.long()), torch.zeros_like(rank))
    place[..., :n] = src
    return now, sums, place, K, V


def _plain_rope(case, x, at, back):
    """Rotated rows, [B, heads, T, d] in order; the angles in 64 bits."""
    rot = case["rot"]
    angle = at.double()[:, None, :, None] * torch.tensor(_freqs(case), dtype=torch.float64, device=x.device)
    c, s = (_gain(case) * torch.cos(angle)).float(), (_gain(case) * torch.sin(angle)).float()
    s = -s if back else s
    f = x.float()
    out = f.clone(memory_format=torch.contiguous_format)
    if case["layout"] == "half":
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    else:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, a * s + b * c
    return out.to(x.dtype)


# ------------------------------------------------------------ what is measured


def prepare(case, seed):
    if case["op"].startswith("rope"):
        Q, K, at = _rope_inputs(case, seed)
        st = dict(case=case, Q=Q, K=K, at=at)
        if own:
            import compressed_attention_adaptive_gb300 as mita
            dt = {"bf16": mita.BF16, "f32": mita.F32}[case["dtype"]]
            flags = mita.FLAG_INTERLEAVED if case["layout"] == "interleaved" else 0
            st["p"] = mita.RopeParams(case["B"], case["H"], case["Hkv"], case["T"], case["d"], case["rot"],
                                      freqs=tuple(_freqs(case)), gain=_gain(case), flags=flags, dtype=dt)
            st["Qo"], st["Ko"] = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (Q, K))
        return st
    x = _cache_inputs(case, seed)
    st = dict(case=case, x=x)
    B, Hkv, d, page = (case[k] for k in ("B", "Hkv", "d", "page"))
    if own:
        import compressed_attention_adaptive_gb300 as mita
        dt = {"bf16": mita.BF16, "f32": mita.F32}[case["dtype"]]
        fill = mita.CacheParams(B, Hkv, Hkv, x["K"].shape[2], d, page, x["n_pages"], x["cols"], dtype=dt)
        st["cache"] = torch.zeros(mita.mita_cache_size(fill), dtype=torch.uint8, device="cuda")
        ws = mita.cache_workspace(fill)
        mita.mita_cache_write(fill, x["K"], x["V"], st["cache"], x["table"], x["lens"], ws, counts=x["lens"],
                              exps=x["exps"])
        mita.mita_device_status(ws)
        st["acc_out"] = torch.zeros_like(x["acc"])
        if case["op"] == "weigh":
            st["p"] = mita.CacheParams(B, case["H"], Hkv, case["T"], d, page, x["n_pages"], x["cols"],
                                       flags=mita.FLAG_CAUSAL if case["causal"] else 0, dtype=dt)
            st["ws"] = mita.cache_workspace(st["p"])
        else:
            most = min(x["K"].shape[2], max(_keeps(case)))
            st["p"] = mita.CacheParams(B, Hkv, Hkv, most, d, page, x["n_pages"], x["cols"], dtype=dt)
            st["ws"], st["read_ws"] = mita.cache_evict_workspace(st["p"]), mita.cache_workspace(st["p"])
            st["len_out"] = torch.empty_like(x["lens"])
            st["src"] = torch.zeros(x["acc"].shape, dtype=torch.int32, device="cuda")
            st["Kr"], st["Vr"] = (torch.zeros((B, Hkv, most, d), dtype=_dtype(case), device="cuda") for _ in range(2))
    else:
        e = x["exps"]
        st["pool"] = (_fill(x, case, x["K"], None if e is None else e[0]),
                      _fill(x, case, x["V"], None if e is None else e[1]))
    del x["K"], x["V"]
    return st


def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        import compressed_attention_adaptive_gb300 as mita
        if op.startswith("rope"):
            call = mita.mita_rope if op == "rope" else mita.mita_rope_backward
            call(st["p"], st["Q"], st["K"], st["Qo"], st["Ko"], pos=st["at"])
            return st["Qo"], st["Ko"]
        x = st["x"]
        if op == "weigh":
            mita.mita_cache_weights(st["p"], x["Q"], st["cache"], x["table"], x["lens"], x["lse"], x["acc"], st["ws"],
                                    counts=x["counts"], exps=x["exps"], decay=case["decay"], acc_out=st["acc_out"])
            return st["acc_out"]
        mita.mita_cache_evict(st["p"], st["cache"], x["table"], x["lens"], x["keep"], x["acc"], st["ws"],
                              first=case["first"], recent=case["recent"], len_out=st["len_out"],
                              acc_out=st["acc_out"], src_out=st["src"])
        mita.mita_cache_read(st["p"], st["cache"], x["table"], st["len_out"], st["Kr"], st["Vr"], st["read_ws"],
                             counts=st["len_out"])
        return st["len_out"], st["acc_out"], st["src"], st["Kr"], st["Vr"]
    if op.startswith("rope"):
        return tuple(_plain_rope(case, st[k], st["at"], op == "rope_back") for k in ("Q", "K"))
    return _plain_weigh(st) if op == "weigh" else _plain_evict(st)


def work(case):
    elem = 2 if case["dtype"] == "bf16" else 4
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"].startswith("rope"):
        rows = B * case["T"] * (case["H"] + Hkv)
        return {"bytes": 2 * rows * d * elem + 4 * B * case["T"], "flops": 3 * rows * case["rot"]}
    lens = _lens(case)
    row = d // 2 + d // 16  # one token's keys, or its values, in the cache
    ints = 4 * sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "weigh":
        counts, H = _counts(case), case["H"]
        seen = sum(sum(n - (c - 1 - t) if case["causal"] else n for t in range(c)) for n, c in zip(lens, counts))
        sums = sum(lens) + (sum(n - c for n, c in zip(lens, counts)) if case["decay"] else 0)
        return {"bytes": sum(lens) * Hkv * row + 4 * Hkv * sums + sum(counts) * H * (d * elem + 4) + ints + 8 * B,
                "flops": 2 * H * d * seen}
    new = [min(n, k) for n, k in zip(lens, _keeps(case))]
    moved = 0.0  # kept rows at or behind the new length, of sums in no order
    for n, k in zip(lens, new):
        if n > k:
            r = min(case["recent"], n - k)
            free = n - case["first"] - case["recent"]
            moved += r + (k - case["first"] - case["recent"]) * max(0, n - case["recent"] - k) / max(1, free)
    # the sums read, kept ones and places written; moved rows; all that is kept read back
    return {"bytes": Hkv * (4 * sum(lens) + 8 * sum(new) + 4 * row * moved + sum(new) * 2 * (row + d * elem))
            + ints + 12 * B, "flops": Hkv * sum(lens)}


# ------------------------------------------- the definition in 64 bits, by itself


def _def_values(x, e):
    """Values in 64 bits that rows x are held as, straight from the format:
    nearest points on the two grids, ties to the even one."""
    y = x.double() * (1.0 if e is None else 2.0 ** -e)
    y = y.reshape(x.shape[:-1] + (-1, 16))
    a = y.abs().amax(-1, keepdim=True) / 6.0
    # the 127 finite e4m3 magnitudes; even positions have an even last bit
    mags = torch.tensor([(i % 8) * 2.0 ** -9 if i < 8 else (8 + i % 8) * 2.0 ** (i // 8 - 10) for i in range(127)],
                        dtype=torch.float64, device=x.device)
    s = _nearest(a, mags)
    grid = torch.tensor(_CODES, dtype=torch.float64, device=x.device)
    r = torch.where(s > 0, y.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    return torch.copysign(_nearest(r, grid) * s, y).reshape(x.shape) * (1.0 if e is None else 2.0 ** e)


def _nearest(a, grid):
    """Nearest element of an ascending grid, ties to the even position."""
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    pick = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))
    return grid[pick]


def _exact_rope(case, seed):
    Q, K, at = _rope_inputs(case, seed)
    sign = -1.0 if case["op"] == "rope_back" else 1.0
    f = torch.tensor(_freqs(case), dtype=torch.float64, device="cuda")
    half, outs = case["rot"] // 2, []
    for x in (Q, K):
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for b in range(x.shape[0]):
            turn = torch.polar(torch.full((1, 1), _gain(case), dtype=torch.float64, device="cuda"),
                               sign * at[b].double()[:, None] * f[None])
            for h in range(x.shape[1]):
                row = x[b, h].double()
                out[b, h] = row
                i = torch.arange(half, device="cuda")
                re, im = (i, i + half) if case["layout"] == "half" else (2 * i, 2 * i + 1)
                z = torch.complex(row[:, re], row[:, im]) * turn
                out[b, h][:, re], out[b, h][:, im] = z.real, z.imag
        outs.append(out)
    return tuple(outs)


def exact(case, seed):
    if case["op"].startswith("rope"):
        return None if case["B"] * (case["H"] + case["Hkv"]) > 20000 else _exact_rope(case, seed)
    x = _cache_inputs(case, seed)
    lens = _lens(case)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    out = torch.zeros(x["acc"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "weigh":
        G = case["H"] // Hkv
        for b, (n, c) in enumerate(zip(lens, _counts(case))):
            for h in range(Hkv):
                e = None if x["exps"] is None else int(x["exps"][0, h])
                k = _def_values(x["K"][b, h, :n], e)
                if case["decay"]:
                    out[b, h, :n - c] = case["decay"] * x["acc"][b, h, :n - c].double()
                for t in range(c):
                    m = n - (c - 1 - t) if case["causal"] else n
                    q, l = x["Q"][b, h * G:(h + 1) * G, t].double(), x["lse"][b, h * G:(h + 1) * G, t].double()
                    out[b, h, :m] += torch.exp(q @ k[:m].T / math.sqrt(d) - l[:, None]).sum(0)
        return out
    keeps = _keeps(case)
    most = min(max(lens), max(keeps))
    K, V = (torch.zeros((B, Hkv, most, d), dtype=torch.float64, device="cuda") for _ in range(2))
    for b, (n, keep) in enumerate(zip(lens, keeps)):
        new = min(n, keep)
        for h in range(Hkv):
            place = torch.arange(n, device="cuda")
            if n > keep:
                first, last = case["first"], n - case["recent"]
                mid = x["acc"][b, h, first:last].double()
                best = torch.sort(-mid, dim=0, stable=True).indices[:keep - first - case["recent"]] + first
                stay = torch.zeros(n, dtype=torch.bool, device="cuda")
                stay[:first] = True
                stay[last:] = True
                stay[best] = True
                place[:new][~stay[:new]] = place[new:][stay[new:]]
            place = place[:new]
            out[b, h, :new] = x["acc"][b, h].double()[place]
            K[b, h, :new], V[b, h, :new] = (_def_values(x[k][b, h], None)[place] for k in ("K", "V"))
    return None, out, None, K, V
