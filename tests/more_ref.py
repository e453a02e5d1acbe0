"""Builders and plain 64-bit references of the calls over block rows that select, weigh, evict and
share (block summaries, scores, selection, gathered weights, eviction, prefix attention)."""
import numpy as np
import torch

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo

BF16, FP4 = echo.BLOCK_BF16, echo.BLOCK_FP4


def pack_rows(fmt, bs, D, k, v):
    """k, v [n][bs][D] bf16 values (float64) -> rows uint8 [n][bytes], and the values they stand for."""
    n = k.shape[0]
    if fmt == BF16:
        both = np.stack([k, v], 1).astype(np.float32)
        return torch.from_numpy(both).bfloat16().view(torch.int16).numpy().reshape(n, -1).view(np.uint8).copy(), k, v
    ns = bs // 16
    (kc, ks), (vc, vs) = ref.quantise(k), ref.quantise(v)
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(n, ns, 8 * D)
    vb = (vc[..., 0::2] | (vc[..., 1::2] << 4)).reshape(n, ns, 2, 8, 8, D // 16).transpose(0, 1, 2, 4, 3, 5).reshape(n, ns, 8 * D)
    s1 = ks.reshape(n, ns, D)
    s2 = vs.reshape(n, ns, 2, 8, D // 16).transpose(0, 1, 2, 4, 3).reshape(n, ns, D)
    rows = np.concatenate([kb, vb, s1, s2], -1).reshape(n, -1).astype(np.uint8)
    return rows, ref.code_values(kc, ks), ref.code_values(vc, vs)


class Cache:
    """Random rows of n_blocks blocks of Hkv heads; k, v [row][bs][D] are what they stand for."""

    def __init__(self, fmt, bs, D, Hkv, n_blocks, g, scale=1.0):
        self.fmt, self.bs, self.D, self.Hkv = fmt, bs, D, Hkv
        n = n_blocks * Hkv
        r = lambda: ref.bf16_round(g.standard_normal((n, bs, D)) * scale)
        self.rows, self.k, self.v = pack_rows(fmt, bs, D, r(), r())

    def spoil(self, row, offs):
        """NaN patterns in the bytes of tokens `offs` of a row."""
        for o in offs:
            for i in ref.token_bytes(self.fmt, self.bs, self.D, int(o)):
                self.rows[row, i] = 0xFF

    def dev(self):
        return torch.from_numpy(self.rows).view(torch.int16).cuda()


def tables(lens, bs, Hkv, g, heads=False, spare=2, gaps=0.0, first=0):
    """A table of scattered blocks that hold `lens` tokens (-1 elsewhere and at gaps), and the blocks
    that the pool needs.  heads: [B][Hkv][n] rows."""
    lens = np.asarray(lens)
    n = max(1, int(-(-max(int(lens.max()), 1) // bs)))
    shape = (len(lens), Hkv, n) if heads else (len(lens), n)
    need = np.broadcast_to((np.arange(n) * bs < lens[:, None])[:, None] if heads else np.arange(n) * bs < lens[:, None], shape).copy()
    need &= g.random(shape) >= gaps
    t = np.full(shape, -1, np.int32)
    total = int(need.sum()) + spare
    t[need] = first + g.permutation(total)[:int(need.sum())]
    return t, total


def row_of(table, Hkv, b, h, i):
    if table.ndim == 3:
        return int(table[b, h, i])
    return int(table[b, i]) * Hkv + h if table[b, i] >= 0 else -1


def tokens_of(cache, table, b, h, n):
    """Keys and values of tokens 0 .. n of (b, h) and which are held: [n][D], [n][D], [n]."""
    k, v, held = np.zeros((n, cache.D)), np.zeros((n, cache.D)), np.zeros(n, bool)
    for i in range(-(-n // cache.bs)):
        r, e = row_of(table, cache.Hkv, b, h, i), min(n, (i + 1) * cache.bs)
        if r >= 0:
            s = slice(i * cache.bs, e)
            k[s], v[s], held[s] = cache.k[r, :e - i * cache.bs], cache.v[r, :e - i * cache.bs], True
    return k, v, held


def select(scores, nb, k, first, last, held):
    """Chosen blocks of one row, ascending, -1 padded."""
    s = np.where(np.isnan(scores), -np.inf, scores)
    cand = [i for i in range(nb) if held[i]]
    must = {i for i in cand if i < first or i >= nb - last}
    order = sorted(cand, key=lambda i: (0 if i in must else 1, -s[i], i))
    out = sorted(order[:k])
    return out + [-1] * (k - len(out))


def evict(acc, pos, n, keep, sinks, recent, nxt):
    """Which slot each of the first min(n, keep) slots takes its token from."""
    if n <= keep:
        return np.arange(n)
    key = np.where(np.isnan(acc[:n]), -np.inf, acc[:n])
    nan = np.isnan(acc[:n])
    must = np.arange(n) < sinks
    if recent:
        must |= pos[:n] >= nxt - recent
    order = sorted(range(n), key=lambda i: (not must[i], nan[i], -key[i], i))
    stay = np.zeros(n, bool)
    stay[order[:keep]] = True
    src = np.arange(keep)
    src[~stay[:keep]] = np.nonzero(stay[keep:])[0] + keep
    return src
