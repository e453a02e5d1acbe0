"""The block-level (GQA) serving operators as measured cases: the tables that name a
request's cache rows, the norm + rotation that fills them, and the attention that reads
them.

A cache row is one block of `bs` tokens of one KV head (keys, then values), either bf16
[2][bs][D] or 4-bit: sub-blocks of 16 tokens, each 18*D bytes --
  key codes [16 tokens][D/2], value codes [2][8][8 tokens][D/16],
  key scales [16 tokens][D/16], value scales [2][D/16][8 tokens]
-- two e2m1 codes a byte (the lower dimension in the low nibble), one e4m3 scale per
token and 16 dimensions.  With a block table shared by the KV heads, block `id` of KV
head `h` is row id * Hkv + h.

Each case runs in a plain form (`own` false: elementary torch operations in 32 bits) or
through the package's calls (`own` true).  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# |x| against s * EDGE[i] decides between code i and i + 1 (a tie takes the even code)
EDGE = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a full batch: each request gets one token, a few a new block
        dict(name="tables_decode", op="tables", B=64, L=32768, new=1, bs=64, done=0),
        # a scheduler step mixing prefill chunks, draft rollbacks and finished requests
        dict(name="tables_mixed", op="tables", B=256, L=8192, new=4096, bs=64, done=16),
        # one request, one token: the smallest call of a decode loop
        dict(name="rope_token", op="rope", T=1, Hq=64, Hkv=8, D=128, rd=128, inter=False, fmt="bf16", bs=64, norm=True),
        # a decode batch into a 4-bit cache, half the dimensions rotated in pairs
        dict(name="rope_decode_fp4", op="rope", T=96, Hq=32, Hkv=8, D=128, rd=64, inter=True, fmt="fp4", bs=64, norm=True),
        # a prefill chunk into a bf16 cache
        dict(name="rope_prefill", op="rope", T=16384, Hq=64, Hkv=8, D=128, rd=128, inter=False, fmt="bf16", bs=64, norm=True),
        # an odd prefill chunk of small heads into a 4-bit cache, no norm
        dict(name="rope_prefill_fp4", op="rope", T=8191, Hq=24, Hkv=8, D=64, rd=64, inter=False, fmt="fp4", bs=32, norm=False),
        # one short chat turn: latency
        dict(name="attn_short", op="attn", B=1, n_q=1, Hq=32, Hkv=8, D=128, L=1000, fmt="bf16", bs=64, sinks=0, window=0, sel=0),
        # the decode batch of the sweep's sizes, bf16 cache, ragged lengths
        dict(name="attn_decode", op="attn", B=16, n_q=1, Hq=64, Hkv=8, D=128, L=32768, fmt="bf16", bs=64, sinks=0, window=0, sel=0),
        # the same batch on a 4-bit cache
        dict(name="attn_decode_fp4", op="attn", B=16, n_q=1, Hq=64, Hkv=8, D=128, L=32768, fmt="fp4", bs=64, sinks=0, window=0, sel=0),
        # streaming decode: a sliding window and four sink tokens, all other blocks gone
        dict(name="attn_window", op="attn", B=64, n_q=1, Hq=64, Hkv=8, D=128, L=131072, fmt="bf16", bs=64, sinks=4, window=4096, sel=0),
        # sixteen recalled blocks of each (request, KV head): the block-sparse step's consumer
        dict(name="attn_recalled", op="attn", B=8, n_q=1, Hq=64, Hkv=8, D=128, L=65536, fmt="bf16", bs=64, sinks=0, window=0, sel=16),
        # long contexts on a 4-bit cache, two query tokens a request (a draft to verify)
        dict(name="attn_long_fp4", op="attn", B=8, n_q=2, Hq=64, Hkv=8, D=128, L=131072, fmt="fp4", bs=64, sinks=0, window=0, sel=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "attn", "attn", "attn"])
    bs = rng.choice([16, 32, 64, 64, 128])
    if op == "tables":
        B = _log(rng, 1, 512)
        L = _log(rng, 100, 32768)
        new = rng.choice([1, 1, 2, _log(rng, 3, 4096)])
        return dict(op="tables", B=B, L=L, new=new, bs=bs, done=rng.randrange(0, B // 4 + 1))
    D = rng.choice([64, 128, 128])
    fmt = rng.choice(["bf16", "fp4"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "rope":
        inter = rng.random() < 0.4
        rd = rng.choice([16, 32, 64, D])
        return dict(op="rope", T=_log(rng, 1, 12000), Hq=Hkv * min(G, 8), Hkv=Hkv, D=D, rd=rd, inter=inter, fmt=fmt,
                    bs=bs, norm=rng.random() < 0.7)
    n_q = rng.choice([1, 1, 1, 2, 3, 4])
    L = _log(rng, 17, 131072)
    B = max(1, min(_log(rng, 1, 64), 4000000 // (L * Hkv)))
    kind = rng.choice(["full", "full", "window", "sel"])
    window = _log(rng, 1, 4096) if kind == "window" else 0
    sinks = rng.choice([0, 1, 4, 17, 64]) if window else 0
    nblk = (L + bs - 1) // bs
    sel = max(1, min(nblk, _log(rng, 1, 64))) if kind == "sel" else 0
    return dict(op="attn", B=B, n_q=n_q, Hq=Hkv * G, Hkv=Hkv, D=D, L=L, fmt=fmt, bs=bs, sinks=sinks, window=window,
                sel=sel)


def _ceil(a, b):
    return (a + b - 1) // b


def _row_bytes(c):
    return c["bs"] * c["D"] * 4 if c["fmt"] == "bf16" else c["bs"] // 16 * 18 * c["D"]


def _tok_bytes(c):
    """Bytes of one token's key and value of one KV head."""
    return c["D"] * 4 if c["fmt"] == "bf16" else c["D"] * 18 // 16


def work(c):
    if c["op"] == "tables":
        old, new = _lengths(c, 0)
        moved = int((-(-new // c["bs"]) - (-(-old // c["bs"]))).abs().sum())
        # lengths in, offsets out; a position and a slot for every entry a step may have
        # (the unused ones get -1); a block id read and written for each block that moves
        return {"bytes": 8 * c["B"] + 4 * (c["B"] + 1) + 8 * c["B"] * c["new"] + 8 * moved, "flops": 0}
    if c["op"] == "rope":
        n_in = (c["Hq"] + 2 * c["Hkv"]) * c["D"] * 2
        n_out = c["Hq"] * c["D"] * 2 + c["Hkv"] * _tok_bytes(c)
        n_out += 2 * c["Hkv"] * c["D"] * 2 if c["fmt"] == "fp4" else 0
        return {"bytes": c["T"] * (n_in + n_out + c["rd"] * 4 + 8), "flops": c["T"] * (c["Hq"] + c["Hkv"]) * c["D"] * 6}
    lens = _ctx(c, 0)
    tokens = int(_visible(c, lens).sum()) * c["Hkv"]
    qo = c["B"] * c["n_q"] * c["Hq"] * c["D"] * 4
    return {"bytes": tokens * _tok_bytes(c) + qo, "flops": tokens * (c["Hq"] // c["Hkv"]) * c["n_q"] * c["D"] * 4}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cpu_gen(seed, k):
    return torch.Generator().manual_seed((seed * 1000003 + k) % (1 << 62))


def _lengths(c, seed):
    """Request lengths before and after a step (int64, CPU): `done` requests end, an eighth
    of the others give back a few draft tokens when chunks are longer than one token, the
    rest grow by up to `new` tokens."""
    g = _cpu_gen(seed, 1)
    B = c["B"]
    old = torch.randint(0, c["L"] + 1, (B,), generator=g)
    grow = torch.full((B,), c["new"]) if c["new"] <= 2 else torch.randint(1, c["new"] + 1, (B,), generator=g)
    new = old + grow
    if c["new"] > 2:
        back = torch.rand(B, generator=g) < 0.125
        new = torch.where(back, (old - torch.randint(1, 9, (B,), generator=g)).clamp(min=0), new)
    if c["done"]:
        new[torch.randperm(B, generator=g)[:c["done"]]] = 0
    return old, new


def _ctx(c, seed):
    """Context lengths, the new tokens included: between half the capacity and all of it
    (at least one token of each query)."""
    g = _cpu_gen(seed, 2)
    lo = max(c["n_q"], c["L"] // 2)
    n = torch.randint(lo, max(lo, c["L"]) + 1, (c["B"],), generator=g)
    n[0] = max(lo, c["L"])
    return n


def _visible(c, lens):
    """Tokens of each request that some query sees."""
    if c["sel"]:
        return torch.full_like(lens, c["sel"] * c["bs"]).minimum(lens)
    if not c["window"]:
        return lens
    return torch.minimum(lens, torch.full_like(lens, c["sinks"] + c["window"] + c["n_q"] - 1))


def _e4m3(x):
    return x.clamp(max=448.0).to(torch.float8_e4m3fn)


def _quantise(x):
    """x [..., D] bf16-valued fp32 -> codes uint8 [..., D], scales e4m3 [..., D/16]."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    s8 = _e4m3(g.abs().amax(-1) / 6.0)
    s = s8.float()[..., None]
    a = g.abs()
    code = torch.zeros_like(g, dtype=torch.uint8)
    for i, e in enumerate(EDGE):
        t = s * e
        code += ((a >= t) if i % 2 else (a > t)).to(torch.uint8)
    code = torch.where(s > 0, code, torch.zeros_like(code)) | ((g < 0).to(torch.uint8) << 3)
    return code.reshape(x.shape), s8


def _pack_rows(k, v, bs, D):
    """k, v [n][bs][D] bf16 -> rows uint8 [n][bs/16*18*D]."""
    n, ns = k.shape[0], bs // 16
    kc, ks = _quantise(k.float())
    vc, vs = _quantise(v.float())
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(n, ns, 8 * D)
    vb = vc[..., 0::2] | (vc[..., 1::2] << 4)                                  # [n][bs][D/2]
    vb = vb.reshape(n, ns, 2, 8, 8, D // 16).permute(0, 1, 2, 4, 3, 5).reshape(n, ns, 8 * D)
    ks = ks.view(torch.uint8).reshape(n, ns, D)
    vs = vs.view(torch.uint8).reshape(n, ns, 2, 8, D // 16).transpose(-1, -2).reshape(n, ns, D)
    return torch.cat([kb, vb, ks, vs], -1).reshape(n, ns * 18 * D)


def _cache_rows(c, n_rows, g):
    """Cache rows of normal keys and values, int16 [n_rows][R]."""
    bs, D = c["bs"], c["D"]
    if c["fmt"] == "bf16":
        return torch.randn(n_rows, 2 * bs * D, generator=g, device="cuda", dtype=torch.bfloat16).view(torch.int16)
    rows = torch.empty(n_rows, bs // 16 * 18 * D, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (bs * D))
    for r in range(0, n_rows, step):
        m = min(step, n_rows - r)
        kv = torch.randn(2, m, bs, D, generator=g, device="cuda", dtype=torch.bfloat16)
        rows[r:r + m] = _pack_rows(kv[0], kv[1], bs, D)
    return rows.view(torch.int16)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    i32 = lambda t: t.to(torch.int32).cuda()
    if c["op"] == "tables":
        old, new = _lengths(c, seed)
        B, bs = c["B"], c["bs"]
        mb = _ceil(c["L"] + c["new"], bs)
        nb_old = -(-old // bs)
        used = int(nb_old.sum())
        n_blocks = B * mb
        perm = torch.randperm(n_blocks, generator=_cpu_gen(seed, 3))
        table = torch.full((B, mb), -1, dtype=torch.int64)
        has = torch.arange(mb)[None] < nb_old[:, None]
        table[has] = perm[:used]
        free = torch.full((n_blocks,), -1, dtype=torch.int64)
        free[:n_blocks - used] = perm[used:]
        s.update(old=i32(old), new=i32(new), table=i32(table), free=i32(free),
                 count=i32(torch.tensor([n_blocks - used])), max_new=B * c["new"])
        return s
    D, bs, Hkv, Hq = c["D"], c["bs"], c["Hkv"], c["Hq"]
    if c["op"] == "rope":
        T, rd = c["T"], c["rd"]
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda", dtype=torch.bfloat16)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["wq"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda") if c["norm"] else None
        s["wk"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda") if c["norm"] else None
        max_pos = 32768
        ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
        s["cs"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        # sequences of consecutive positions, their blocks scattered over the cache
        cg = _cpu_gen(seed, 4)
        nseq = max(1, min(T, 8 if T > 512 else T))
        start = torch.randint(0, max_pos - _ceil(T, nseq) - bs, (nseq,), generator=cg)
        t = torch.arange(T)
        seq, at = t % nseq, t // nseq
        order = torch.argsort(seq, stable=True)
        seq, at = seq[order], at[order]
        pos = start[seq] + at
        blk = at + start[seq] % bs
        per = _ceil(_ceil(T, nseq) + bs, bs)
        ids = torch.randperm(nseq * per, generator=cg).reshape(nseq, per)
        s["slot"] = i32(ids[seq, blk // bs] * bs + blk % bs)
        s["pos"] = i32(pos)
        s["rows"] = torch.zeros(nseq * per * Hkv, _row_bytes(c) // 2, dtype=torch.int16, device="cuda")
        return s
    B, n_q, L = c["B"], c["n_q"], c["L"]
    lens = _ctx(c, seed)
    nblk = _ceil(L, bs)
    s["q"] = torch.randn(B, n_q, Hq, D, generator=g, device="cuda", dtype=torch.bfloat16)
    s["ctx"] = i32(lens)
    s["scale"] = D ** -0.5
    cg = _cpu_gen(seed, 5)
    if c["sel"]:
        # each (request, KV head) has its own blocks, at scattered rows of the pool
        pick = torch.rand(B, Hkv, nblk, generator=cg)
        pick = torch.where(torch.arange(nblk) * bs < lens[:, None, None], pick, torch.full((), -1.0))
        top = pick.topk(c["sel"], -1)
        sel = torch.where(top.values >= 0, top.indices, torch.full((), nblk, dtype=torch.int64)).sort(-1).values
        sel = torch.where(sel < nblk, sel, torch.full((), -1, dtype=torch.int64))
        rows = torch.randperm(B * Hkv * c["sel"], generator=cg).reshape(B, Hkv, c["sel"])
        s["sel"], s["table"] = i32(sel), i32(torch.where(sel >= 0, rows, torch.full((), -1, dtype=torch.int64)))
        n_rows = B * Hkv * c["sel"]
    else:
        at = torch.arange(nblk) * bs
        need = at < lens[:, None]
        if c["window"]:   # only the blocks that some query sees are held
            need &= (at < c["sinks"]) | (at + bs > (lens - (n_q - 1) - c["window"])[:, None])
        n = int(need.sum())
        table = torch.full((B, nblk), -1, dtype=torch.int64)
        table[need] = torch.randperm(n, generator=cg)
        s["sel"], s["table"], n_rows = None, i32(table), n * Hkv
    s["rows"] = _cache_rows(c, n_rows, g)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_tables(s):
    c, old, new = s["case"], s["old"].long(), s["new"].long()
    bs, dev = c["bs"], old.device
    nb_old, nb_new = (old + bs - 1) // bs, (new + bs - 1) // bs
    freed, grown, tok = (nb_old - nb_new).clamp(min=0), (nb_new - nb_old).clamp(min=0), (new - old).clamp(min=0)
    table, free, n0 = s["table"].clone(), s["free"].clone(), s["count"].long()
    ex = lambda x: x.cumsum(0) - x
    b_f = torch.repeat_interleave(torch.arange(c["B"], device=dev), freed)
    i_f = torch.arange(b_f.numel(), device=dev)
    free[n0 + i_f] = table[b_f, nb_new[b_f] + i_f - ex(freed)[b_f]]
    top = n0 + freed.sum()
    b_g = torch.repeat_interleave(torch.arange(c["B"], device=dev), grown)
    i_g = torch.arange(b_g.numel(), device=dev)
    at = top - 1 - i_g
    table[b_g, nb_old[b_g] + i_g - ex(grown)[b_g]] = torch.where(at >= 0, free[at.clamp(min=0)], -1)
    count = (top - grown.sum()).clamp(min=0).to(torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), tok.cumsum(0)])
    b_t = torch.repeat_interleave(torch.arange(c["B"], device=dev), tok)
    p = old[b_t] + torch.arange(b_t.numel(), device=dev) - cu[b_t]
    blk = table[b_t, p // bs].long()
    slot = torch.full((s["max_new"],), -1, dtype=torch.int32, device=dev)
    pos = slot.clone()
    slot[:b_t.numel()] = torch.where(blk >= 0, blk * bs + p % bs, -1).to(torch.int32)
    pos[:b_t.numel()] = p.to(torch.int32)
    return {"table": table, "free": free, "count": count, "slot": slot, "pos": pos, "cu": cu.to(torch.int32)}


def _rotate(x, cs, rd, inter):
    """x [T][H][D]; cs [T][rd] (cosines, then sines)."""
    cos, sin = cs[:, None, :rd // 2], cs[:, None, rd // 2:]
    r = x[..., :rd]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rd // 2], r[..., rd // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([r, x[..., rd:]], -1)


def _plain_norm(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def _values(codes, scales):
    """codes uint8 [..., D], scales e4m3 [..., D/16] -> the values they stand for, fp32."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    v = lut.index_select(0, codes.flatten().int()).reshape(*codes.shape[:-1], -1, 16)
    return (v * scales.float()[..., None]).reshape(codes.shape)


def _plain_rope(s):
    c = s["case"]
    T, Hkv, D, bs = c["T"], c["Hkv"], c["D"], c["bs"]
    cs = s["cs"][s["pos"].long()]
    q = _rotate(_plain_norm(s["q"], s["wq"]), cs, c["rd"], c["inter"]).bfloat16()
    k = _rotate(_plain_norm(s["k"], s["wk"]), cs, c["rd"], c["inter"]).bfloat16()
    slot = s["slot"].long()
    row = (slot // bs)[:, None] * Hkv + torch.arange(Hkv, device=slot.device)
    off = (slot % bs)[:, None].expand(T, Hkv)
    if c["fmt"] == "bf16":
        rows = s["rows"].view(torch.bfloat16).view(-1, 2, bs, D)
        rows[row, 0, off] = k
        rows[row, 1, off] = s["v"]
        return {"q": q, "rows": s["rows"].view(torch.bfloat16)}
    kc, ks = _quantise(k.float())
    vc, vs = _quantise(s["v"].float())
    rows = s["rows"].view(torch.uint8).view(-1, bs // 16, 18 * D)
    sub, t = off // 16, off % 16
    rows[..., :8 * D].unflatten(-1, (16, D // 2))[row, sub, t] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    rows[..., 8 * D:16 * D].unflatten(-1, (2, 8, 8, D // 16))[row, sub, t // 8, :, t % 8] = \
        (vc[..., 0::2] | (vc[..., 1::2] << 4)).unflatten(-1, (8, D // 16))
    rows[..., 16 * D:17 * D].unflatten(-1, (16, D // 16))[row, sub, t] = ks.view(torch.uint8)
    rows[..., 17 * D:].unflatten(-1, (2, D // 16, 8))[row, sub, t // 8, :, t % 8] = vs.view(torch.uint8)
    # what the cache now holds for these tokens, as the values it stands for
    return {"q": q, "k": _values(kc, ks).bfloat16(), "v": _values(vc, vs).bfloat16()}


def _tokens(s):
    """The cache tokens a plain pass looks at: their positions [B][1 or Hkv][S], rows
    [B][Hkv][S] (-1: not held), offsets, and which of them are listed once."""
    c, table, lens = s["case"], s["table"].long(), s["ctx"].long()
    bs, Hkv, dev = c["bs"], c["Hkv"], table.device
    heads = torch.arange(Hkv, device=dev)[None, :, None]
    if c["sel"]:
        sel = s["sel"].long()
        off = torch.arange(bs, device=dev).repeat(sel.shape[-1])[None, None]
        pos = sel.repeat_interleave(bs, -1) * bs + off
        row = table.repeat_interleave(bs, -1)
        return pos, torch.where(pos >= 0, row, -1), off.expand_as(pos), pos >= 0
    if c["window"]:
        w0 = (lens - c["window"] - (c["n_q"] - 1))[:, None]
        first = torch.arange(c["sinks"], device=dev)[None].expand(c["B"], -1)
        last = w0 + torch.arange(c["window"] + c["n_q"] - 1, device=dev)
        pos = torch.cat([first, last], 1)[:, None]
        once = torch.cat([first >= 0, last >= c["sinks"]], 1)[:, None] & (pos >= 0) & (pos < lens[:, None, None])
    else:
        pos = torch.arange(c["L"], device=dev)[None, None].expand(c["B"], 1, -1)
        once = pos < lens[:, None, None]
    p = torch.where(once, pos, 0)
    ids = table.gather(1, (p // bs)[:, 0])[:, None]
    row = torch.where(ids >= 0, ids * Hkv + heads, -1)
    return pos, row, (p % bs).expand_as(row), once


def _plain_kv(s, row, off):
    c = s["case"]
    bs, D = c["bs"], c["D"]
    row = row.clamp(min=0)
    if c["fmt"] == "bf16":
        rows = s["rows"].view(torch.bfloat16).view(-1, 2, bs, D)
        return rows[row, 0, off].float(), rows[row, 1, off].float()
    rows = s["rows"].view(torch.uint8).view(-1, bs // 16, 18 * D)
    sub, t = off // 16, off % 16
    kb = rows[..., :8 * D].unflatten(-1, (16, D // 2))[row, sub, t]
    vb = rows[..., 8 * D:16 * D].unflatten(-1, (2, 8, 8, D // 16))[row, sub, t // 8, :, t % 8].flatten(-2)
    ks = rows[..., 16 * D:17 * D].unflatten(-1, (16, D // 16))[row, sub, t].view(torch.float8_e4m3fn)
    vs = rows[..., 17 * D:].unflatten(-1, (2, D // 16, 8))[row, sub, t // 8, :, t % 8].contiguous()
    code = lambda b: torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return _values(code(kb), ks), _values(code(vb), vs.view(torch.float8_e4m3fn))


def _plain_attn(s):
    c, lens = s["case"], s["ctx"].long()
    B, n_q, Hq, Hkv, D = c["B"], c["n_q"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    pos, row, off, once = _tokens(s)
    k, v = _plain_kv(s, row, off)
    q = s["q"].float().view(B, n_q, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n_q * G, D)
    x = (q @ k.transpose(-1, -2)).view(B, Hkv, n_q, G, -1) * s["scale"]
    seen = lens[:, None] - (n_q - 1 - torch.arange(n_q, device=lens.device))             # [B][n_q]
    seen = seen[:, None, :, None, None]
    p = pos[:, :, None, None]
    ok = (p < seen) & (once & (row >= 0))[:, :, None, None]
    if c["window"]:
        ok &= (p < c["sinks"]) | (p >= seen - c["window"])
    x = x.masked_fill(~ok, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - m.masked_fill(m == -math.inf, 0.0)).exp()
    l = e.sum(-1, keepdim=True)
    o = (e.view(B, Hkv, n_q * G, -1) @ v).view(B, Hkv, n_q, G, D) / l.masked_fill(l == 0, 1.0)
    lse = (m + l.log())[..., 0]
    return {"out": o.transpose(1, 2).reshape(B, n_q, Hq, D).bfloat16(),
            "lse": lse.transpose(1, 2).reshape(B, n_q, Hq)}


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _own_plan(s):
    """The argument block, outputs and workspace that a serving loop keeps."""
    import sparse_attention_kv_fp8_gb300 as echo
    c = s["case"]
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")
    bf16 = lambda *n: torch.empty(n, dtype=torch.bfloat16, device="cuda")
    if c["op"] == "tables":
        out = {"table": s["table"], "free": s["free"], "count": i32(1), "slot": i32(s["max_new"]),
               "pos": i32(s["max_new"]), "cu": i32(c["B"] + 1)}
        args = echo.make_block_tables_args(s["old"], s["new"], c["bs"], s["table"], s["free"], s["count"],
                                           out["count"], out["slot"], out["pos"], out["cu"], dev_status=s["status"])
        return echo.echo_block_tables, args, out
    fmt = echo.BLOCK_BF16 if c["fmt"] == "bf16" else echo.BLOCK_FP4
    if c["op"] == "rope":
        T, Hkv, D = c["T"], c["Hkv"], c["D"]
        out = {"q": bf16(T, c["Hq"], D)}
        if c["fmt"] == "fp4":
            out.update(k=bf16(T, Hkv, D), v=bf16(T, Hkv, D))
        args = echo.make_qk_norm_rope_args(s["q"], s["k"], s["v"], s["pos"], s["cs"], out["q"], q_weight=s["wq"],
                                           k_weight=s["wk"], eps=1e-6, interleaved=c["inter"], slot_map=s["slot"],
                                           rows=s["rows"], fmt=fmt, block_tokens=c["bs"], k_out=out.get("k"),
                                           v_out=out.get("v"), dev_status=s["status"])
        if c["fmt"] == "bf16":
            out["rows"] = s["rows"].view(torch.bfloat16)
        return echo.echo_qk_norm_rope, args, out
    out = {"out": bf16(c["B"], c["n_q"], c["Hq"], c["D"]),
           "lse": torch.empty(c["B"], c["n_q"], c["Hq"], dtype=torch.float32, device="cuda")}
    ws = echo.BlockAttentionWorkspace(c["n_q"] * (c["Hq"] // c["Hkv"]), c["D"])
    args = echo.make_block_attention_args(s["q"], s["rows"], s["table"], s["ctx"], c["Hkv"], s["scale"], out["out"],
                                          out["lse"], ws, fmt=fmt, block_tokens=c["bs"], sel=s["sel"],
                                          sinks=c["sinks"], window=c["window"], dev_status=s["status"])
    return echo.echo_block_attention, args, out


def run(s):
    if own:
        if "plan" not in s:
            s["plan"] = _own_plan(s)
        call, args, out = s["plan"]
        call(args)
        return out
    return {"tables": _plain_tables, "rope": _plain_rope, "attn": _plain_attn}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_code(x):
    """The 4-bit value of each entry of x [..., 16k] (bf16-valued): the nearest multiple
    of the group's scale on the e2m1 grid, ties to the even code."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    g = x.double().unflatten(-1, (-1, 16))
    s = _e4m3((g.abs().amax(-1) / 6.0).float()).double()[..., None]
    t = torch.where(s > 0, g.abs() / s.clamp(min=1e-9), 0.0)
    hi = torch.bucketize(t, grid).clamp(max=7)             # the first grid value >= t
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - t, t - grid[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (grid[code] * s * g.sign()).flatten(-2)


def _exact_rope(s):
    c = s["case"]
    rd, n = c["rd"], c["rd"] // 2
    ang = s["cs"][s["pos"].long()].double()[:, None]

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
        i = torch.arange(n, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if c["inter"] else (i, i + n)
        y = x.clone()
        y[..., ia] = x[..., ia] * ang[..., :n] - x[..., ib] * ang[..., n:]
        y[..., ib] = x[..., ib] * ang[..., :n] + x[..., ia] * ang[..., n:]
        return y

    q, k = one(s["q"], s["wq"]), one(s["k"], s["wk"])
    if c["fmt"] == "fp4":
        return {"q": q, "k": _exact_code(k.to(torch.bfloat16)), "v": _exact_code(s["v"])}
    T, Hkv, D, bs = c["T"], c["Hkv"], c["D"], c["bs"]
    rows = torch.zeros(s["rows"].shape[0] // Hkv, Hkv, 2, bs, D, dtype=torch.float64, device=q.device)
    blk, off = s["slot"].long() // bs, s["slot"].long() % bs
    rows[blk, :, 0, off] = k
    rows[blk, :, 1, off] = s["v"].double()
    return {"q": q, "rows": rows.view(s["rows"].shape[0], -1)}


def _exact_block(s, r):
    """Keys and values [n][bs][D] of rows r [n] in 64 bits."""
    c = s["case"]
    bs, D = c["bs"], c["D"]
    x = s["rows"][r]
    if c["fmt"] == "bf16":
        x = x.view(torch.bfloat16).double().view(-1, 2, bs, D)
        return x[:, 0], x[:, 1]
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=r.device)
    b = x.view(torch.uint8).view(-1, 18 * D)               # one sub-block of 16 tokens a row
    f8 = lambda y: y.contiguous().view(torch.float8_e4m3fn).double()
    both = lambda y: torch.stack([grid[(y & 15).long()], grid[(y >> 4).long()]], -1).flatten(-2)
    k = both(b[:, :8 * D].reshape(-1, 16, D // 2)).unflatten(-1, (-1, 16)) * f8(b[:, 16 * D:17 * D]).view(-1, 16, D // 16, 1)
    v = both(b[:, 8 * D:16 * D].reshape(-1, 2, 8, 8, D // 16)).transpose(2, 3).reshape(-1, 16, D // 16, 16)
    v = v * f8(b[:, 17 * D:]).view(-1, 2, D // 16, 8).transpose(2, 3).reshape(-1, 16, D // 16, 1)
    return k.reshape(-1, bs, D), v.reshape(-1, bs, D)


def _exact_attn(s):
    c, bs = s["case"], s["case"]["bs"]
    B, n_q, Hq, Hkv, D = c["B"], c["n_q"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    if B * Hkv > 600:
        return None
    out = torch.zeros(B, n_q, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, n_q, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens, table = s["ctx"].tolist(), s["table"].long()
    sel = s["sel"].long() if s["sel"] is not None else None
    for b in range(B):
        for h in range(Hkv):
            if sel is not None:
                lb, r = sel[b, h], table[b, h]
            else:
                lb = torch.arange(table.shape[1], device="cuda")
                r = torch.where(table[b] >= 0, table[b] * Hkv + h, -1)
            held = (r >= 0) & (lb >= 0)
            lb, r = lb[held], r[held]
            k, v = _exact_block(s, r)
            p = (lb[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
            k, v = k.reshape(-1, D), v.reshape(-1, D)
            for j in range(n_q):
                n = lens[b] - (n_q - 1 - j)
                see = p < n
                if c["window"]:
                    see &= (p < c["sinks"]) | (p >= n - c["window"])
                if not bool(see.any()):
                    continue
                x = s["q"][b, j, h * G:(h + 1) * G].double() @ k[see].T * s["scale"]
                lse[b, j, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[b, j, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v[see]
    return {"out": out, "lse": lse}


def exact(c, seed):
    if c["op"] == "tables":      # whole numbers only
        return None
    s = prepare(c, seed)
    return _exact_rope(s) if c["op"] == "rope" else _exact_attn(s)
