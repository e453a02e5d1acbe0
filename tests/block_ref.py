"""Plain 64-bit references of the block calls, on the CPU, and builders of block rows.

Rows are handled as bytes; `Cache` keeps a GPU array of rows and the tokens' exact values
side by side."""
import math

import numpy as np
import torch

import sparse_attention_kv_fp8_gb300 as echo

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(b & 128, -v, v)
    v[127] = v[255] = np.nan
    return v


E4M3 = e4m3_values()


def nearest_even(x, grid):
    """Index of the value of `grid` (ascending, >= 0) nearest to x >= 0, ties to the even index."""
    hi = np.minimum(np.searchsorted(grid, x), grid.size - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - x, x - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise(x):
    """x [..., 16k] of bf16 values (float64) -> codes [..., 16k], scale bytes [..., k]: the
    definition, in 64 bits (amax / 6 rounded to fp32 first, as the kernel's division is)."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    a = np.abs(g)
    amax = a.max(-1)
    s = nearest_even(np.minimum((amax.astype(np.float32) / np.float32(6)).astype(np.float64), 448.0), E4M3[:127])
    sv = E4M3[s][..., None]
    code = np.where(sv > 0, nearest_even(np.minimum(a / np.where(sv > 0, sv, 1.0), 6.0), GRID), 0)
    code = code | ((g < 0) << 3)
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def code_values(codes, scales):
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    return (v.reshape(*codes.shape[:-1], -1, 16) * E4M3[scales][..., None]).reshape(codes.shape)


def token_bytes(fmt, bs, D, off):
    """Byte places, inside a row, of one token's key and value: (key, value) index arrays
    for bf16; (key codes, key scales, value codes, value scales) for 4-bit."""
    if fmt == echo.BLOCK_BF16:
        k = off * D * 2 + np.arange(2 * D)
        return k, bs * D * 2 + k
    base, t = off // 16 * 18 * D, off % 16
    vb = base + 8 * D + (t // 8) * 4 * D
    parts = np.arange(8)[:, None] * 8 + t % 8
    vc = (vb + parts * (D // 16) + np.arange(D // 16)).reshape(-1)
    vs = base + 17 * D + (t // 8) * (D // 2) + np.arange(D // 16) * 8 + t % 8
    return (base + t * (D // 2) + np.arange(D // 2), base + 16 * D + t * (D // 16) + np.arange(D // 16), vc, vs)


def bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint8)


def bf16_round(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().double().numpy()


def write_token(row, fmt, bs, D, off, k, v):
    """Writes k, v [D] (bf16 values) as token `off` of the byte row; returns what it stands for."""
    if fmt == echo.BLOCK_BF16:
        ki, vi = token_bytes(fmt, bs, D, off)
        row[ki], row[vi] = bf16_bits(k), bf16_bits(v)
        return k, v
    (kc, ks), (vc, vs) = quantise(k), quantise(v)
    a, b, c, d = token_bytes(fmt, bs, D, off)
    row[a], row[b] = kc[0::2] | (kc[1::2] << 4), ks
    row[c], row[d] = vc[0::2] | (vc[1::2] << 4), vs
    return code_values(kc, ks), code_values(vc, vs)


def read_token(row, fmt, bs, D, off):
    if fmt == echo.BLOCK_BF16:
        ki, vi = token_bytes(fmt, bs, D, off)
        f = lambda i: torch.from_numpy(row[i].copy()).view(torch.bfloat16).double().numpy()
        return f(ki), f(vi)
    a, b, c, d = token_bytes(fmt, bs, D, off)
    both = lambda x: np.stack([x & 15, x >> 4], -1).reshape(-1)
    return code_values(both(row[a]), row[b]), code_values(both(row[c]), row[d])


def attention(q, tokens, scale):
    """q [M][D], tokens: list over the M rows of (k [n][D], v [n][D]); float64 softmax.
    Returns out [M][D], lse [M], and for the error bounds: sum of softmax * |v| [M][D], the
    largest sum |q_d k_d| * scale [M], max |q| * largest sum |k_d| * scale [M], sum |v| [M][D]."""
    M, D = q.shape
    out, lse, av, sv = np.zeros((M, D)), np.full(M, -np.inf), np.zeros((M, D)), np.zeros((M, D))
    mag, tiny = np.zeros(M), np.zeros(M)
    for i, (k, v) in enumerate(tokens):
        if not len(k):
            continue
        x = k @ q[i] * scale
        m = x.max()
        e = np.exp(x - m)
        out[i], lse[i], av[i] = e @ v / e.sum(), m + math.log(e.sum()), e @ np.abs(v) / e.sum()
        mag[i] = (np.abs(k) @ np.abs(q[i])).max() * abs(scale)
        tiny[i] = np.abs(k).sum(1).max() * np.abs(q[i]).max() * abs(scale)
        sv[i] = np.abs(v).sum(0)
    return out, lse, av, mag, tiny, sv


def attention_bounds(fmt, D, n, out, lse, av, mag, tiny, sv):
    """How far fp32 arithmetic with 16-bit softmax weights may be from 64 bits.

    A score is a sum of D products in fp32 (each addition off by 2^-24 of the partial sum, at
    most sum |q_d k_d|), plus two more roundings for its scaling; 4-bit rows take the queries
    to fp16 on a grid of 2^-25 of the row's largest.  A score off by d moves every weight by a
    factor 1 +- 2 d (numerator and denominator).  Weights are rounded to 16 bits (half a step:
    bf16 2^-8, fp16 2^-11; fp16 weights, kept at 2^7 times their value relative to a running
    maximum that is at most the true one, so that the sum of weights is at least 2^7, have an
    absolute half step of 2^-25 once subnormal: 2^-32 of the sum each); the value sums add n products in fp32; the output is rounded to
    bf16 (2^-8)."""
    d = (D + 4) * 2.0 ** -24 * mag + (2.0 ** -25 * tiny if fmt == echo.BLOCK_FP4 else 0.0) + 2.0 ** -22
    u = 2.0 ** -11 if fmt == echo.BLOCK_FP4 else 2.0 ** -8
    rel = u + 2.5 * d + (n + 16) * 2.0 ** -24
    far = 2.0 ** -8 * np.abs(out) + rel[..., None] * av * (1 + 2.0 ** -7)
    far = far + (2.0 ** -32 * sv if fmt == echo.BLOCK_FP4 else 0.0)
    with np.errstate(invalid="ignore"):
        far_lse = d + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0) + (n + 16) * 2.0 ** -24 + 2.0 ** -22
    return far, far_lse


def norm_rope(x, w, eps, cs, rd, inter):
    """x [T][H][D], cs [T][rd]; float64.  Returns y and the magnitude its error scales with."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    n = rd // 2
    c, s = cs[:, None, :n], cs[:, None, n:]
    i = np.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + n)
    y, mag = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = np.abs(a * c) + np.abs(b * s)
    mag[..., ib] = np.abs(b * c) + np.abs(a * s)
    return y, mag


def block_tables(old, new, bs, table, free, count, max_new):
    """The definition, one block at a time.  Returns (table, free, count, slot, pos, cu,
    len_out, exhausted)."""
    table, stack = table.copy(), list(free[:count])
    B, nb = len(old), lambda n: -(-n // bs)
    for b in range(B):
        for i in range(nb(new[b]), nb(old[b])):
            stack.append(table[b, i])
    top, need, ok = len(stack), 0, np.ones(B, bool)
    free = free.copy()
    free[count:top] = stack[count:]
    for b in range(B):
        grow = max(0, nb(new[b]) - nb(old[b]))
        need += grow
        if grow and need > top:
            ok[b] = False
            continue
        for i in range(nb(old[b]), nb(new[b])):
            table[b, i] = stack.pop()
    slot, pos, cu = np.full(max_new, -1, np.int32), np.full(max_new, -1, np.int32), [0]
    for b in range(B):
        for p in range(old[b], new[b]):
            i = cu[-1] + p - old[b]
            if ok[b] and i < max_new:
                slot[i], pos[i] = table[b, p // bs] * bs + p % bs, p
        cu.append(cu[-1] + max(0, new[b] - old[b]))
    return table, free, len(stack), slot, pos, np.array(cu, np.int32), np.where(ok, new, old), not ok.all()


def two_term_bounds(D, n, out, lse, av, mag, tiny, sv):
    """attention_bounds of bf16 rows for softmax weights that enter the value product as two bf16
    terms: what the first leaves out is at most 2^-8 of the weight, and the second is off by at
    most 2^-8 of that, 2^-16 of the weight in all (a single term: 2^-8).  The product adds 2 n
    terms, 16 at a time, each addition off by up to 2^-23 (the tensor cores cut off)."""
    d = (D + 4) * 2.0 ** -24 * mag + 2.0 ** -22
    rel = 2.0 ** -16 + 2.5 * d + (4 * n + 64) * 2.0 ** -24
    return 2.0 ** -8 * np.abs(out) + rel[..., None] * av * (1 + 2.0 ** -7)


def opposite_values(g, n, D):
    """n tokens' values [n][D] (bf16), each odd token the negative of the one before it: with near
    equal weights their sum is far below its terms."""
    v = bf16_round(g.uniform(2, 4, (n, D)) * g.choice([-1.0, 1.0], (n, D)))
    v[1::2] = -v[0:n - n % 2:2]
    return v
