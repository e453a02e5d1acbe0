"""More block-level serving operators as measured cases: block summaries, their scores
and the selection that block-sparse attention reads; attention of requests that share a
prefix; the weights that tokens gather and the eviction that goes by them.

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
EDGE = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
INF = math.inf


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode step's last blocks: every request got one token, its block is summed up anew
        dict(name="summary_decode", op="summary", B=64, L=4096, new=1, Hkv=8, D=128, fmt="bf16", bs=64),
        # prompts just written: all of their blocks
        dict(name="summary_prompt", op="summary", B=8, L=16384, new=0, Hkv=8, D=128, fmt="bf16", bs=64),
        # one request, one token: latency
        dict(name="scores_token", op="scores", B=1, n_q=1, Hq=32, Hkv=8, D=128, L=4000, bs=64, gaps=False),
        # long contexts, two query tokens a request (a draft to verify), some blocks gone
        dict(name="scores_long", op="scores", B=16, n_q=2, Hq=64, Hkv=8, D=128, L=131072, bs=64, gaps=True),
        # sixteen blocks of each (request, KV head) of a decode step
        dict(name="select_decode", op="select", B=8, n_q=1, Hkv=8, L=65536, bs=64, k=16, first=1, last=2, gaps=False),
        # a prefill chunk, each of its queries with blocks of its own
        dict(name="select_chunk", op="select", B=1, n_q=1000, Hkv=8, L=65536, bs=64, k=32, first=1, last=2, gaps=True),
        # short contexts in 4 bits: latency
        dict(name="weights_short", op="weights", B=4, n_q=1, Hq=32, Hkv=8, D=128, L=1100, fmt="fp4", bs=32, decay=0.99),
        # the decode batch of the attention's sizes
        dict(name="weights_long", op="weights", B=16, n_q=1, Hq=64, Hkv=8, D=128, L=32768, fmt="bf16", bs=64, decay=1.0),
        # a cache at its budget: a step's new tokens push as many old ones out
        dict(name="evict_step", op="evict", B=32, L=4100, new=4, keep=4096, sinks=4, recent=256, Hkv=8, D=128, fmt="bf16", bs=64),
        # prompts cut down to the budget
        dict(name="evict_prompt", op="evict", B=8, L=32768, new=32768, keep=4096, sinks=4, recent=512, Hkv=8, D=128, fmt="bf16", bs=64),
        # a few answers sampled from one prompt
        dict(name="prefix_samples", op="prefix", B=4, n_q=1, Hq=32, Hkv=8, D=128, P=1000, L=100, groups=1, fmt="bf16", bs=64),
        # a full batch behind one long document
        dict(name="prefix_document", op="prefix", B=64, n_q=1, Hq=64, Hkv=8, D=128, P=32768, L=1000, groups=1, fmt="bf16", bs=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["summary", "scores", "select", "weights", "weights", "evict", "prefix", "prefix", "prefix"])
    bs = rng.choice([16, 32, 48, 64, 64, 128])
    D = rng.choice([64, 128, 128])
    fmt = rng.choice(["bf16", "fp4"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    n_q = rng.choice([1, 1, 1, 2, 3, 4])
    if op == "summary":
        L = _log(rng, 17, 32768)
        B = max(1, min(_log(rng, 1, 64), 1000000 // (L * Hkv)))
        return dict(op=op, B=B, L=L, new=rng.choice([0, 1, 2, _log(rng, 3, 4096)]), Hkv=Hkv, D=D, fmt=fmt, bs=bs)
    if op == "scores":
        L = _log(rng, 17, 131072)
        B = max(1, min(_log(rng, 1, 64), 16000000 // (L * Hkv)))
        return dict(op=op, B=B, n_q=n_q, Hq=Hkv * G, Hkv=Hkv, D=D, L=L, bs=bs, gaps=rng.random() < 0.5)
    if op == "select":
        L = _log(rng, 17, 131072)
        rows = max(1, min(_log(rng, 1, 2048), 8000000 * bs // (L * Hkv * 64)))
        n_q = rng.choice([1, n_q, rows])
        first, last = rng.choice([(0, 0), (1, 1), (1, 2), (0, 3)])
        k = max(first + last, 1, _log(rng, 1, 128))
        return dict(op=op, B=max(1, rows // n_q), n_q=n_q, Hkv=Hkv, L=L, bs=bs, k=k, first=first, last=last,
                    gaps=rng.random() < 0.5)
    if op == "weights":
        L = _log(rng, 17, 65536)
        B = max(1, min(_log(rng, 1, 64), 3000000 // (L * Hkv)))
        return dict(op=op, B=B, n_q=n_q, Hq=Hkv * G, Hkv=Hkv, D=D, L=L, fmt=fmt, bs=bs, decay=rng.choice([1.0, 0.99, 0.5]))
    if op == "evict":
        L = _log(rng, 33, 32768)
        B = max(1, min(_log(rng, 1, 64), 2000000 // (L * Hkv)))
        keep = max(8, L - _log(rng, 1, L))
        sinks, recent = rng.choice([(0, 0), (4, 0), (1, keep // 4), (4, keep // 2)])
        return dict(op=op, B=B, L=L, new=rng.choice([1, 4, max(1, L // 8), L]), keep=keep, sinks=sinks, recent=recent,
                    Hkv=Hkv, D=D, fmt=fmt, bs=bs)
    P = _log(rng, 16, 32768)
    B = max(2, min(_log(rng, 2, 64), 100000000 // (P * Hkv * G * n_q)))
    L = max(n_q, min(_log(rng, 1, 4096), 500000 // (B * Hkv)))
    return dict(op=op, B=B, n_q=n_q, Hq=Hkv * G, Hkv=Hkv, D=D, P=P, L=L, groups=rng.choice([1, 1, 2, min(5, B)]), fmt=fmt,
                bs=bs)


def _ceil(a, b):
    return (a + b - 1) // b


def _row_bytes(c):
    return c["bs"] * c["D"] * 4 if c["fmt"] == "bf16" else c["bs"] // 16 * 18 * c["D"]


def _key_bytes(c):
    """Bytes of one token's key of one KV head (its value takes as many)."""
    return c["D"] * 2 if c["fmt"] == "bf16" else c["D"] * 9 // 16


def work(c):
    op = c["op"]
    if op == "summary":
        lens = _ctx(c, 0)
        start = _old(c, lens) // c["bs"]
        tokens = int((lens - start * c["bs"]).sum()) * c["Hkv"]
        blocks = int((_ceil(lens, c["bs"]) - start).sum())
        return {"bytes": tokens * _key_bytes(c) + blocks * (c["Hkv"] * c["D"] * 4 + 4), "flops": 2 * tokens * c["D"]}
    if op == "scores":
        blocks = int(_ceil(_ctx(c, 0), c["bs"]).sum()) * c["Hkv"]
        qb = c["B"] * c["n_q"] * c["Hq"] * c["D"] * 2
        return {"bytes": blocks * (c["D"] * 4 + 4 * c["n_q"]) + qb,
                "flops": blocks * c["n_q"] * (c["Hq"] // c["Hkv"]) * c["D"] * 4}
    if op == "select":
        rows = c["B"] * c["n_q"] * c["Hkv"]
        blocks = int(_ceil(_ctx(c, 0), c["bs"]).sum()) * c["n_q"] * c["Hkv"]
        return {"bytes": 4 * blocks + 8 * rows * c["k"], "flops": 0}
    if op == "weights":
        tokens = int(_ctx(c, 0).sum()) * c["Hkv"]
        qb = c["B"] * c["n_q"] * c["Hq"] * (c["D"] * 2 + 4)
        return {"bytes": tokens * (_key_bytes(c) + 8) + qb, "flops": tokens * c["n_q"] * (c["Hq"] // c["Hkv"]) * c["D"] * 2}
    if op == "evict":
        lens = _ctx(c, 0)
        over = lens > c["keep"]
        # every token's weight is read; the kept tokens' weights and positions are written;
        # of the tokens past the budget those that are kept move: of evenly mixed weights
        # (len - keep) * keep / len
        n = lens.double()
        moved = float(torch.where(over, (n - c["keep"]) * c["keep"] / n, 0.0).sum()) * c["Hkv"]
        kept = int(lens.clamp(max=c["keep"]).sum()) * c["Hkv"]
        return {"bytes": int(lens.sum()) * c["Hkv"] * 4 + kept * 8 + int(moved * 4 * _key_bytes(c)), "flops": 0}
    plen, own_len, start = _shared(c, 0)
    G = c["Hq"] // c["Hkv"]
    n = start[1:] - start[:-1]
    tokens = int(plen.sum() + own_len.sum()) * c["Hkv"]
    pairs = int((plen * n).sum() + own_len.sum()) * c["Hq"] * c["n_q"]
    return {"bytes": tokens * 2 * _key_bytes(c) + c["B"] * c["n_q"] * c["Hq"] * c["D"] * 4, "flops": pairs * c["D"] * 4}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cpu_gen(seed, k):
    return torch.Generator().manual_seed((seed * 1000003 + k) % (1 << 62))


def _ctx(c, seed):
    """Context lengths, the new tokens included: between half the capacity and all of it
    (at least one token of each query); near the budget where a cache is kept at one."""
    g = _cpu_gen(seed, 2)
    lo = max(c.get("n_q", 1), c["L"] // 2)
    if c["op"] == "evict" and c["new"] < c["L"] // 2:
        lo = c["L"] - c["new"]
    n = torch.randint(min(lo, c["L"]), max(lo, c["L"]) + 1, (c["B"],), generator=g)
    n[0] = max(lo, c["L"])
    return n


def _old(c, lens):
    return torch.zeros_like(lens) if c["new"] == 0 else (lens - c["new"]).clamp(min=0)


def _shared(c, seed):
    """Prefix lengths of the groups, own lengths of the requests, the groups' first
    requests (the last request of a larger batch shares nothing)."""
    g = _cpu_gen(seed, 6)
    n, B = c["groups"], c["B"]
    plen = torch.randint(max(1, c["P"] // 2), c["P"] + 1, (n,), generator=g)
    plen[0] = c["P"]
    end = B - 1 if B > 8 else B
    cuts = torch.randperm(end - 1, generator=g)[:n - 1].sort().values + 1 if n > 1 else torch.zeros(0, dtype=torch.int64)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([end])])
    own_len = torch.randint(c["n_q"], max(c["n_q"], c["L"]) + 1, (B,), generator=g)
    return plen, own_len, start


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
    vb = vc[..., 0::2] | (vc[..., 1::2] << 4)
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


def _table(need, cg, base=0):
    """Scattered ids of a pool's blocks where `need` [B][n], -1 elsewhere; the pool's size."""
    t = torch.full(need.shape, -1, dtype=torch.int64)
    t[need] = base + torch.randperm(need.numel(), generator=cg)[:int(need.sum())]
    return t, need.numel()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cg = _cpu_gen(seed, 5)
    s = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    i32 = lambda t: t.to(torch.int32).cuda()
    randn = lambda *n: torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16)
    op, B, bs, Hkv, L = c["op"], c["B"], c["bs"], c["Hkv"], c["L"]
    D = c.get("D", 0)
    if op == "prefix":
        plen, own_len, start = _shared(c, seed)
        at = torch.arange(_ceil(c["P"], bs)) * bs
        ptab, n0 = _table(at < plen[:, None], cg)
        at = torch.arange(_ceil(max(L, c["n_q"]), bs)) * bs
        table, n1 = _table(at < own_len[:, None], cg, n0)
        s.update(plen=i32(plen), ptab=i32(ptab), start=i32(start), ctx=i32(own_len), table=i32(table), scale=D ** -0.5,
                 q=randn(B, c["n_q"], c["Hq"], D), rows=_cache_rows(c, (n0 + n1) * Hkv, g),
                 groups=start.tolist())
        return s
    lens = _ctx(c, seed)
    nblk = _ceil(max(L, c.get("n_q", 1)), bs)
    need = torch.arange(nblk) * bs < lens[:, None]
    if c.get("gaps"):       # blocks that were given back
        need &= torch.rand(B, nblk, generator=cg) > 0.05
    table, n = _table(need, cg)
    s.update(ctx=i32(lens), table=i32(table))
    if op == "summary":
        s.update(old=i32(_old(c, lens)), rows=_cache_rows(c, n * Hkv, g),
                 summary=torch.zeros(n * Hkv, 2, D, dtype=torch.bfloat16, device="cuda"))
    elif op == "scores":
        mid, half = randn(n * Hkv, D), 0.5 + randn(n * Hkv, D).abs()
        s.update(q=randn(B, c["n_q"], c["Hq"], D), scale=D ** -0.5, summary=torch.stack([mid - half, mid + half], 1))
    elif op == "select":
        # scores of a bound's spread, a part of them on a coarse grid (equal ones among them)
        x = 3.0 + torch.randn(B, c["n_q"], Hkv, nblk, generator=g, device="cuda")
        coarse = torch.rand(B, c["n_q"], Hkv, 1, generator=g, device="cuda") < 0.25
        x = torch.where(coarse, (x * 8).round() / 8, x)
        s["scores"] = torch.where((s["table"] >= 0)[:, None, None], x, torch.full((), -INF, device="cuda"))
    elif op == "weights":
        n_q, Hq = c["n_q"], c["Hq"]
        q = randn(B, n_q, Hq, D)
        # log sum exp of scores against normal keys: log n + variance / 2
        var = (q.float() * D ** -0.5).square().sum(-1)
        seen = (s["ctx"][:, None] - (n_q - 1) + torch.arange(n_q, device="cuda")).clamp(min=1)
        s.update(q=q, scale=D ** -0.5, rows=_cache_rows(c, n * Hkv, g), lse=seen.float().log()[..., None] + var / 2,
                 old=i32((lens - n_q).clamp(min=0)),
                 acc=torch.empty(B, Hkv, nblk * bs, device="cuda").exponential_(generator=g) * 0.01)
    else:
        T = nblk * bs
        acc = torch.randn(B, Hkv, T, generator=g, device="cuda").exp()
        acc[torch.rand(B, Hkv, T, generator=g, device="cuda") < 0.1] = 0.0      # tokens nobody looked at
        old = (lens - c["new"]).clamp(min=0)
        # the older tokens come from anywhere in a context that is longer than the cache
        nxt = lens + torch.where(old > 0, torch.randint(0, 4096, (B,), generator=cg), 0)
        pos = torch.zeros(B, 1, T, dtype=torch.int64)
        for b in range(B):
            m = int(old[b])
            pos[b, 0, :m] = torch.randperm(int(nxt[b]) - int(lens[b]) + m, generator=cg)[:m]
        s.update(acc=acc, pos=i32(pos.expand(B, Hkv, T).contiguous()), pos_len=i32(old), next_pos=i32(nxt),
                 rows=_cache_rows(c, n * Hkv, g))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _values(codes, scales):
    """codes uint8 [..., D], scales e4m3 [..., D/16] -> the values they stand for, fp32."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    v = lut.index_select(0, codes.flatten().int()).reshape(*codes.shape[:-1], -1, 16)
    return (v * scales.float()[..., None]).reshape(codes.shape)


def _plain_k(c, rows, row, off):
    """Keys [...][D] of tokens (row, off), fp32."""
    bs, D = c["bs"], c["D"]
    if c["fmt"] == "bf16":
        return rows.view(torch.bfloat16).view(-1, 2, bs, D)[row, 0, off].float()
    r = rows.view(torch.uint8).view(-1, bs // 16, 18 * D)
    sub, t = off // 16, off % 16
    b = r[..., :8 * D].unflatten(-1, (16, D // 2))[row, sub, t]
    sc = r[..., 16 * D:17 * D].unflatten(-1, (16, D // 16))[row, sub, t].view(torch.float8_e4m3fn)
    return _values(torch.stack([b & 15, b >> 4], -1).flatten(-2), sc)


def _plain_v(c, rows, row, off):
    bs, D = c["bs"], c["D"]
    if c["fmt"] == "bf16":
        return rows.view(torch.bfloat16).view(-1, 2, bs, D)[row, 1, off].float()
    r = rows.view(torch.uint8).view(-1, bs // 16, 18 * D)
    sub, t = off // 16, off % 16
    b = r[..., 8 * D:16 * D].unflatten(-1, (2, 8, 8, D // 16))[row, sub, t // 8, :, t % 8].flatten(-2)
    sc = r[..., 17 * D:].unflatten(-1, (2, D // 16, 8))[row, sub, t // 8, :, t % 8].contiguous()
    return _values(torch.stack([b & 15, b >> 4], -1).flatten(-2), sc.view(torch.float8_e4m3fn))


def _where_tokens(table, bs, Hkv, S):
    """Row [B][Hkv][S] (0 where not held), offset and held [B][1][S] of tokens 0 .. S."""
    p = torch.arange(S, device=table.device)
    ids = table.long()[:, None, p // bs]
    row = ids.clamp(min=0) * Hkv + torch.arange(Hkv, device=table.device)[:, None]
    return row, (p % bs).expand_as(row), ids >= 0


def _plain_summary(s):
    c, bs, Hkv = s["case"], s["case"]["bs"], s["case"]["Hkv"]
    lens, old = s["ctx"].long(), s["old"].long()
    blk = torch.arange(s["table"].shape[1], device="cuda")
    b, i = ((blk >= (old // bs)[:, None]) & (blk * bs < lens[:, None])).nonzero(as_tuple=True)
    row = (s["table"].long()[b, i][:, None] * Hkv + torch.arange(Hkv, device="cuda"))           # [n][Hkv]
    off = torch.arange(bs, device="cuda")
    k = _plain_k(c, s["rows"], row[..., None].expand(-1, -1, bs), off.expand(*row.shape, bs))     # [n][Hkv][bs][D]
    seen = (i * bs)[:, None] + off < lens[b][:, None]
    seen = seen[:, None, :, None]
    s["summary"][row, 0] = k.masked_fill(~seen, INF).amin(2).bfloat16()
    s["summary"][row, 1] = k.masked_fill(~seen, -INF).amax(2).bfloat16()
    return s["summary"]


def _seen(s):
    """Tokens each query sees [B][n_q]."""
    n_q = s["case"]["n_q"]
    return s["ctx"].long()[:, None] - (n_q - 1 - torch.arange(n_q, device="cuda"))


def _plain_scores(s):
    c = s["case"]
    B, n_q, Hq, Hkv, D, bs = c["B"], c["n_q"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    ids = s["table"].long()
    n = ids.shape[1]
    row = ids.clamp(min=0)[:, None] * Hkv + torch.arange(Hkv, device="cuda")[:, None]
    lo, hi = s["summary"][row].float().unbind(-2)
    q = s["q"].float().view(B, n_q, Hkv, Hq // Hkv, D).transpose(1, 2).reshape(B, Hkv, -1, D) * s["scale"]
    x = q.clamp(min=0) @ hi.transpose(-1, -2) + q.clamp(max=0) @ lo.transpose(-1, -2)
    x = x.view(B, Hkv, n_q, Hq // Hkv, n).amax(3).transpose(1, 2)                                # [B][n_q][Hkv][n]
    ok = (torch.arange(n, device="cuda") * bs < _seen(s)[..., None]) & (ids >= 0)[:, None]
    return x.masked_fill(~ok[:, :, None], -INF)


def _plain_select(s):
    c = s["case"]
    B, n_q, Hkv, bs, k = c["B"], c["n_q"], c["Hkv"], c["bs"], c["k"]
    ids = s["table"].long()
    n = ids.shape[1]
    seen = _seen(s)
    i, nb = torch.arange(n, device="cuda"), ((seen + bs - 1) // bs)[..., None]
    ok = ((i < nb) & (ids >= 0)[:, None])[:, :, None]                                            # [B][n_q][1][n]
    must = ((i < c["first"]) | (i >= nb - c["last"]))[:, :, None]
    x = torch.where(must, INF, s["scores"]).masked_fill(~ok, -INF)
    # (a chosen block of score -inf comes before one that may not be chosen)
    order = x.sort(dim=-1, descending=True, stable=True).indices
    may = ok.expand_as(x).gather(-1, order)
    order = order.gather(-1, may.to(torch.uint8).sort(dim=-1, descending=True, stable=True).indices)[..., :k]
    good = ok.expand_as(x).gather(-1, order)
    sel = torch.where(good, order, n).sort(-1).values
    sel = torch.where(sel < n, sel, -1)
    if sel.shape[-1] < k:
        sel = torch.nn.functional.pad(sel, (0, k - sel.shape[-1]), value=-1)
    rows = ids[:, None, None].expand(B, n_q, Hkv, n).gather(-1, sel.clamp(min=0)) * Hkv + \
        torch.arange(Hkv, device="cuda")[:, None]
    rows = torch.where(sel >= 0, rows, -1)
    return {"sel": sel.int(), "rows": rows.int(), "len": seen.clamp(min=0).int()}


def _plain_weights(s):
    c = s["case"]
    B, n_q, Hq, Hkv, D = c["B"], c["n_q"], c["Hq"], c["Hkv"], c["D"]
    S = s["acc"].shape[-1]
    row, off, held = _where_tokens(s["table"], c["bs"], Hkv, S)
    k = _plain_k(c, s["rows"], row, off)
    q = s["q"].float().view(B, n_q, Hkv, Hq // Hkv, D).transpose(1, 2).reshape(B, Hkv, -1, D) * s["scale"]
    lse = s["lse"].view(B, n_q, Hkv, -1).transpose(1, 2).reshape(B, Hkv, -1, 1)
    w = (q @ k.transpose(-1, -2) - lse).exp().view(B, Hkv, n_q, Hq // Hkv, S).sum(3)
    p = torch.arange(S, device="cuda")
    ok = (p < _seen(s)[..., None])[:, None] & held[:, :, None]
    w = w.masked_fill(~ok, 0.0).sum(2)
    before = torch.where(p < s["old"].long()[:, None], s["acc"].transpose(0, 1) * c["decay"], 0.0).transpose(0, 1)
    return torch.where((p < s["ctx"].long()[:, None])[:, None], before + w, 0.0)


def _move(c, rows, src, dst):
    """Copies tokens (row, offset) src to dst in place."""
    bs, D = c["bs"], c["D"]
    (r0, o0), (r1, o1) = src, dst
    if c["fmt"] == "bf16":
        x = rows.view(-1, 2, bs, D)
        x[r1, :, o1] = x[r0, :, o0]
        return
    x = rows.view(torch.uint8).view(-1, bs // 16, 18 * D)
    a, t, b, u = o0 // 16, o0 % 16, o1 // 16, o1 % 16
    for part, shape in ((x[..., :8 * D], (16, D // 2)), (x[..., 16 * D:17 * D], (16, D // 16))):
        y = part.unflatten(-1, shape)
        y[r1, b, u] = y[r0, a, t]
    y = x[..., 8 * D:16 * D].unflatten(-1, (2, 8, 8, D // 16))
    y[r1, b, u // 8, :, u % 8] = y[r0, a, t // 8, :, t % 8]
    y = x[..., 17 * D:].unflatten(-1, (2, D // 16, 8))
    y[r1, b, u // 8, :, u % 8] = y[r0, a, t // 8, :, t % 8]


def _plain_evict(s):
    c = s["case"]
    B, Hkv, bs, keep = c["B"], c["Hkv"], c["bs"], c["keep"]
    lens, acc = s["ctx"].long()[:, None, None], s["acc"]
    T = acc.shape[-1]
    p = torch.arange(T, device="cuda").expand(B, Hkv, T)
    nxt = s["next_pos"].long()[:, None, None]
    pos = torch.where(p < s["pos_len"].long()[:, None, None], s["pos"].long(), nxt - lens + p)
    must = (p < c["sinks"]) | (pos >= nxt - c["recent"])
    x = torch.where(must, INF, acc).masked_fill(p >= lens, -INF)
    order = x.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros(B, Hkv, T, dtype=torch.bool, device="cuda").scatter_(-1, order[..., :keep], True) & (p < lens)
    end = lens.clamp(max=keep)
    hole, mover = ~kept & (p < end), kept & (p >= keep)
    dst = torch.where(hole, p, T).sort(-1).values
    src = torch.where(mover, p, T).sort(-1).values
    at = torch.where(p < end, p, T)                 # whose token a slot gets
    at = torch.cat([at, at.new_zeros(B, Hkv, 1)], -1).scatter_(-1, dst, src)[..., :T]
    out = at.clamp(max=T - 1)
    have = p < end
    res = {"acc": torch.where(have, acc.gather(-1, out), 0.0),
           "pos": torch.where(have, pos.gather(-1, out), 0).int(), "len": end[:, 0, 0].int()}
    b, h, i = (dst < T).nonzero(as_tuple=True)
    d, f = dst[b, h, i], src[b, h, i]
    tab = s["table"].long()
    _move(c, s["rows"], (tab[b, f // bs] * Hkv + h, f % bs), (tab[b, d // bs] * Hkv + h, d % bs))
    res["rows"] = s["rows"]
    return res


def _plain_prefix(s):
    c = s["case"]
    B, n_q, Hq, Hkv, D, bs = c["B"], c["n_q"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    G = Hq // Hkv
    q = s["q"].float().view(B, n_q, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n_q * G, D) * s["scale"]
    S = s["table"].shape[1] * bs
    row, off, held = _where_tokens(s["table"], bs, Hkv, S)
    k, v = _plain_k(c, s["rows"], row, off), _plain_v(c, s["rows"], row, off)
    ok = (torch.arange(S, device="cuda") < _seen(s)[..., None])[:, None] & held[:, :, None]       # [B][1][n_q][S]
    x = (q @ k.transpose(-1, -2)).masked_fill(~ok.repeat_interleave(G, 2), -INF)
    top = x.amax(-1, keepdim=True)
    parts = []
    for g in range(c["groups"]):
        b0, b1 = s["groups"][g], s["groups"][g + 1]
        n = s["ptab"].shape[1] * bs
        row, off, held = _where_tokens(s["ptab"][g:g + 1], bs, Hkv, n)
        kp, vp = _plain_k(c, s["rows"], row[0], off[0]), _plain_v(c, s["rows"], row[0], off[0])
        y = q[b0:b1].transpose(0, 1).reshape(Hkv, -1, D) @ kp.transpose(-1, -2)
        y = y.masked_fill(~((torch.arange(n, device="cuda") < s["plen"][g]) & held[0]), -INF)
        y = y.view(Hkv, b1 - b0, n_q * G, n)
        parts.append((b0, b1, y, vp))
        top[b0:b1] = torch.maximum(top[b0:b1], y.amax(-1, keepdim=True).transpose(0, 1))
    top = top.masked_fill(top == -INF, 0.0)
    e = (x - top).exp()
    l, o = e.sum(-1, keepdim=True), e @ v
    for b0, b1, y, vp in parts:
        e = (y - top[b0:b1].transpose(0, 1)).exp()
        l[b0:b1] += e.sum(-1, keepdim=True).transpose(0, 1)
        o[b0:b1] += (e.view(Hkv, -1, y.shape[-1]) @ vp).view(Hkv, b1 - b0, n_q * G, D).transpose(0, 1)
    o = o / l.masked_fill(l == 0, 1.0)
    lse = (top + l.log())[..., 0]
    return {"out": o.view(B, Hkv, n_q, G, D).transpose(1, 2).reshape(B, n_q, Hq, D).bfloat16(),
            "lse": lse.view(B, Hkv, n_q, G).transpose(1, 2).reshape(B, n_q, Hq)}


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _own_plan(s):
    """The argument block, outputs and workspace that a serving loop keeps."""
    import sparse_attention_kv_fp8_gb300 as echo
    c = s["case"]
    op, B, Hkv, bs, st = c["op"], c["B"], c["Hkv"], c["bs"], s["status"]
    fmt = echo.BLOCK_FP4 if c.get("fmt") == "fp4" else echo.BLOCK_BF16
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    if op == "summary":
        args = echo.make_block_summary_args(s["rows"], s["table"], s["ctx"], Hkv, s["summary"], old_len=s["old"],
                                            fmt=fmt, block_tokens=bs, dev_status=st)
        return echo.echo_block_summary, args, s["summary"]
    if op == "scores":
        out = torch.full((B, c["n_q"], Hkv, s["table"].shape[1]), -INF, device="cuda")
        args = echo.make_block_scores_args(s["q"], s["summary"], s["table"], s["ctx"], Hkv, s["scale"], out,
                                           block_tokens=bs, dev_status=st)
        return echo.echo_block_scores, args, out
    if op == "select":
        n_q, k = c["n_q"], c["k"]
        out = {"sel": i32(B, n_q, Hkv, k), "rows": i32(B, n_q, Hkv, k), "len": i32(B, n_q)}
        args = echo.make_block_select_args(s["scores"], s["ctx"], out["sel"], block_tokens=bs, first=c["first"],
                                           last=c["last"], table=s["table"], sel_rows=out["rows"], len_out=out["len"])
        return echo.echo_block_select, args, out
    if op == "weights":
        out = torch.zeros_like(s["acc"])
        args = echo.make_block_weights_args(s["q"], s["rows"], s["table"], s["ctx"], Hkv, s["scale"], s["lse"], s["acc"],
                                            out, old_len=s["old"], decay=c["decay"], fmt=fmt, block_tokens=bs,
                                            dev_status=st)
        return echo.echo_block_weights, args, out
    if op == "evict":
        out = {"acc": torch.zeros_like(s["acc"]), "pos": torch.zeros_like(s["pos"]), "len": i32(B), "rows": s["rows"]}
        ws = echo.BlockEvictWorkspace(B, Hkv, c["keep"])
        args = echo.make_block_evict_args(s["rows"], s["table"], s["ctx"], out["len"], Hkv, c["keep"], s["acc"],
                                          out["acc"], ws, sinks=c["sinks"], recent=c["recent"], pos=s["pos"],
                                          pos_out=out["pos"], pos_len=s["pos_len"], next_pos=s["next_pos"], fmt=fmt,
                                          block_tokens=bs, dev_status=st)
        return echo.echo_block_evict, args, out
    n_q, Hq, D = c["n_q"], c["Hq"], c["D"]
    out = {"out": torch.empty(B, n_q, Hq, D, dtype=torch.bfloat16, device="cuda"),
           "lse": torch.empty(B, n_q, Hq, dtype=torch.float32, device="cuda")}
    ws = echo.PrefixAttentionWorkspace(B, n_q, Hq, Hkv, D)
    args = echo.make_prefix_attention_args(s["q"], s["rows"], s["ptab"], s["plen"], s["start"], s["table"], s["ctx"], Hkv,
                                           s["scale"], out["out"], out["lse"], ws, fmt=fmt, block_tokens=bs,
                                           dev_status=st)
    return echo.echo_prefix_attention, args, out


def run(s):
    if own:
        if "plan" not in s:
            s["plan"] = _own_plan(s)
        call, args, out = s["plan"]
        call(args)
        return out
    return {"summary": _plain_summary, "scores": _plain_scores, "select": _plain_select, "weights": _plain_weights,
            "evict": _plain_evict, "prefix": _plain_prefix}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(c, rows, ids):
    """Keys and values [n * bs][D] of the cache rows `ids` [n], in order."""
    bs, D = c["bs"], c["D"]
    x = rows[ids]
    if c["fmt"] == "bf16":
        x = x.view(torch.bfloat16).double().view(-1, 2, bs, D)
        return x[:, 0].reshape(-1, D), x[:, 1].reshape(-1, D)
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    b = x.view(torch.uint8).view(-1, 18 * D)               # one sub-block of 16 tokens a row
    f8 = lambda y: y.contiguous().view(torch.float8_e4m3fn).double()
    both = lambda y: torch.stack([grid[(y & 15).long()], grid[(y >> 4).long()]], -1).flatten(-2)
    k = both(b[:, :8 * D].reshape(-1, 16, D // 2)).unflatten(-1, (-1, 16)) * f8(b[:, 16 * D:17 * D]).view(-1, 16, D // 16, 1)
    v = both(b[:, 8 * D:16 * D].reshape(-1, 2, 8, 8, D // 16)).transpose(2, 3).reshape(-1, 16, D // 16, 16)
    v = v * f8(b[:, 17 * D:]).view(-1, 2, D // 16, 8).transpose(2, 3).reshape(-1, 16, D // 16, 1)
    return k.reshape(-1, D), v.reshape(-1, D)


def _exact_summary(s):
    c, bs, Hkv = s["case"], s["case"]["bs"], s["case"]["Hkv"]
    out = s["summary"].double()
    for b, (n, m) in enumerate(zip(s["ctx"].tolist(), s["old"].tolist())):
        i0, i1 = m // bs, _ceil(n, bs)
        for h in range(Hkv):
            ids = s["table"][b, i0:i1].long() * Hkv + h
            k = _exact_rows(c, s["rows"], ids)[0]
            lo, hi = k.clone(), k.clone()
            lo[n - i0 * bs:], hi[n - i0 * bs:] = INF, -INF
            out[ids, 0], out[ids, 1] = lo.view(i1 - i0, bs, -1).amin(1), hi.view(i1 - i0, bs, -1).amax(1)
    return out


def _exact_scores(s):
    c, bs, Hkv, n_q = s["case"], s["case"]["bs"], s["case"]["Hkv"], s["case"]["n_q"]
    G = c["Hq"] // Hkv
    out = torch.full((c["B"], n_q, Hkv, s["table"].shape[1]), -INF, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["ctx"].tolist()):
        for h in range(Hkv):
            for j in range(n_q):
                ids = s["table"][b, :_ceil(n - (n_q - 1 - j), bs)].long()
                at = (ids >= 0).nonzero()[:, 0]
                lo, hi = s["summary"][ids[at] * Hkv + h].double().unbind(1)
                for q in s["q"][b, j, h * G:(h + 1) * G].double() * s["scale"]:
                    out[b, j, h, at] = torch.maximum(out[b, j, h, at], torch.maximum(q * lo, q * hi).sum(-1))
    return out


def _exact_weights(s):
    c, bs, Hkv, n_q = s["case"], s["case"]["bs"], s["case"]["Hkv"], s["case"]["n_q"]
    G = c["Hq"] // Hkv
    out = torch.zeros(s["acc"].shape, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(s["ctx"].tolist(), s["old"].tolist())):
        for h in range(Hkv):
            k = _exact_rows(c, s["rows"], s["table"][b, :_ceil(n, bs)].long() * Hkv + h)[0]
            out[b, h, :m] = s["acc"][b, h, :m].double() * c["decay"]
            for j in range(n_q):
                e = n - (n_q - 1 - j)
                x = s["q"][b, j, h * G:(h + 1) * G].double() @ k[:e].T * s["scale"]
                out[b, h, :e] += (x - s["lse"][b, j, h * G:(h + 1) * G, None].double()).exp().sum(0)
    return out


def _exact_prefix(s):
    c, bs, Hkv, n_q = s["case"], s["case"]["bs"], s["case"]["Hkv"], s["case"]["n_q"]
    G, B = c["Hq"] // Hkv, c["B"]
    out = torch.zeros(B, n_q, c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.full((B, n_q, c["Hq"]), -INF, dtype=torch.float64, device="cuda")
    plen, ctx = s["plen"].tolist(), s["ctx"].tolist()
    for h in range(Hkv):
        shared = [tuple(x[:n] for x in _exact_rows(c, s["rows"], s["ptab"][g, :_ceil(n, bs)].long() * Hkv + h))
                  for g, n in enumerate(plen)]
        for b in range(B):
            k, v = _exact_rows(c, s["rows"], s["table"][b, :_ceil(ctx[b], bs)].long() * Hkv + h)
            for j in range(n_q):
                e = ctx[b] - (n_q - 1 - j)
                kj, vj = k[:e], v[:e]
                for g in range(c["groups"]):
                    if s["groups"][g] <= b < s["groups"][g + 1]:
                        kj, vj = torch.cat([shared[g][0], kj]), torch.cat([shared[g][1], vj])
                x = s["q"][b, j, h * G:(h + 1) * G].double() @ kj.T * s["scale"]
                lse[b, j, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[b, j, h * G:(h + 1) * G] = torch.softmax(x, -1) @ vj
    return {"out": out, "lse": lse}


def exact(c, seed):
    if c["op"] in ("select", "evict"):      # whole numbers and moved values only
        return None
    s = prepare(c, seed)
    return {"summary": _exact_summary, "scores": _exact_scores, "weights": _exact_weights,
            "prefix": _exact_prefix}[c["op"]](s)
