"""echo_block_weights (64-bit sums within a derived tolerance) and echo_block_evict (exact, moved rows
byte for byte) on the GPU."""
import numpy as np
import pytest
import torch

import block_ref as ref
import more_ref as mr
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev

pytestmark = pytest.mark.gpu
BF16, FP4 = echo.BLOCK_BF16, echo.BLOCK_FP4
i32 = lambda x: dev(np.array(x, np.int32))
status = lambda: torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# gathered weights
# ---------------------------------------------------------------------------

def check_weights(fmt, D, bs, Hq, Hkv, n_q, lens, old=None, decay=1.0, acc=True, in_place=False, heads=False, gaps=0.0, scale=None,
                  k_shift=0, seed=0):
    g = np.random.default_rng(seed)
    B, G = len(lens), Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    table, n = mr.tables(lens, bs, Hkv, g, heads=heads, gaps=gaps)
    c = mr.Cache(fmt, bs, D, Hkv, n if not heads else -(-n // Hkv), g, scale=2.0 ** k_shift)
    T = table.shape[-1] * bs
    q = ref.bf16_round(g.standard_normal((B, n_q, Hq, D)))
    lse = np.full((B, n_q, Hq), -np.inf)
    before = g.random((B, Hkv, T)).astype(np.float32)
    want, tol = np.full((B, Hkv, T), 55.0), np.zeros((B, Hkv, T))
    for b, m in enumerate(lens):
        for h in range(Hkv):
            k, _, held = mr.tokens_of(c, table, b, h, m)
            k = k * 2.0 ** -k_shift
            o = m if old is None else min(old[b], m)
            if acc:
                want[b, h, :m] = np.where(np.arange(m) < o, before[b, h, :m].astype(np.float64) * np.float32(decay), 0.0)
            else:
                want[b, h, :m] = 0.0
            tol[b, h, :m] = 2.0 ** -23 * np.abs(want[b, h, :m]) * 2
            for j in range(n_q):
                e = max(0, m - (n_q - 1 - j))
                for hq in range(h * G, (h + 1) * G):
                    ok = held[:e]
                    if not ok.any():
                        continue
                    x = k[:e] @ q[b, j, hq] * scale
                    lse[b, j, hq] = np.float32(np.log(np.exp(x[ok] - x[ok].max()).sum()) + x[ok].max())
                    w = np.where(ok, np.exp(x - lse[b, j, hq]), 0.0)
                    want[b, h, :e] += w
                    # the score in fp32 (D products, the tensor cores cut off: 2^-23 each), 4-bit rows take the
                    # query to a grid of 2^-25 of its largest entry; its product with scale log2 e and lse log2 e
                    # rounded (2^-22 of each); the exponential 2^-22; sums of n_q G + 1 terms
                    mag = np.abs(k[:e]) @ np.abs(q[b, j, hq]) * abs(scale)
                    d = (D + 4) * 2.0 ** -23 * mag + 2.0 ** -22 * (np.abs(x) + abs(lse[b, j, hq]) + 1)
                    if fmt == FP4:
                        d = d + 2.0 ** -25 * np.abs(k[:e]).sum(1) * np.abs(q[b, j, hq]).max() * abs(scale)
                    tol[b, h, :e] += w * (1.1 * d + (n_q * G + 1) * 2.0 ** -23)
            for i in range(m // bs, table.shape[-1]):          # tokens past the length: NaN patterns
                r = mr.row_of(table, Hkv, b, h, i)
                if r >= 0:
                    c.spoil(r, range(max(0, m - i * bs), bs))
    qd = torch.from_numpy(q.astype(np.float32)).bfloat16().cuda()
    a = torch.from_numpy(before).cuda() if acc else None
    out = a if in_place else torch.full((B, Hkv, T), 55.0, device="cuda")
    st = status()
    echo.echo_block_weights(echo.make_block_weights_args(
        qd, c.dev(), dev(table), i32(lens), Hkv, scale, torch.from_numpy(lse.astype(np.float32)).cuda(), a, out,
        old_len=i32(old) if old is not None else None, decay=decay, fmt=fmt, block_tokens=bs, k_shift=k_shift, dev_status=st))
    got = out.double().cpu().numpy()
    assert int(st) == 0
    for b, m in enumerate(lens):
        assert (np.abs(got[b, :, :m] - want[b, :, :m]) <= tol[b, :, :m] + 1e-37).all(), (b, np.abs(got[b, :, :m] - want[b, :, :m]).max())
        rest = got[b, :, m:]
        assert (rest == (before[b, :, m:] if in_place else 55.0)).all()      # left as they were


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D,bs", [(128, 64), (64, 16), (128, 48), (64, 128)])
@pytest.mark.parametrize("Hq,Hkv,n_q", [(8, 1, 1), (3, 3, 2), (10, 2, 4), (16, 1, 7)])
def test_weights(fmt, D, bs, Hq, Hkv, n_q):
    check_weights(fmt, D, bs, Hq, Hkv, n_q, [0, 1, 2, 15, 16, 17, 100, 300], decay=0.9)


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_weights_variants(fmt):
    check_weights(fmt, 128, 32, 8, 2, 1, [70, 33], acc=False, seed=1)
    check_weights(fmt, 128, 32, 8, 2, 3, [70, 33, 5], old=[67, 0, 9], decay=0.5, seed=2)
    check_weights(fmt, 64, 32, 8, 2, 2, [70, 33], in_place=True, seed=3)
    check_weights(fmt, 64, 16, 8, 2, 2, [130, 47], heads=True, gaps=0.3, seed=4)
    check_weights(fmt, 64, 16, 2, 2, 1, [40], scale=-0.2, seed=5)
    check_weights(fmt, 64, 16, 2, 2, 1, [40], scale=0.0, seed=6)
    check_weights(fmt, 128, 16, 100, 1, 2, [90, 31], seed=7)         # 200 query rows of a KV head: in four goes
    check_weights(fmt, 128, 64, 16, 2, 1, [5000, 2100], seed=8)


def test_weights_of_shifted_keys():
    check_weights(FP4, 128, 32, 8, 2, 1, [70, 33], k_shift=6, seed=9)


def test_weights_sum_to_the_rows_that_attend():
    """With the lse that the attention returned: each query row hands out a weight of one."""
    g = np.random.default_rng(10)
    lens, bs, Hkv, Hq, D = [700, 20], 64, 2, 8, 128
    for fmt in (BF16, FP4):
        table, n = mr.tables(lens, bs, Hkv, g)
        rows = mr.Cache(fmt, bs, D, Hkv, n, g).dev()
        q = torch.from_numpy(g.standard_normal((2, 1, Hq, D)).astype(np.float32)).bfloat16().cuda()
        out, lse, ws = torch.empty_like(q), torch.empty(2, 1, Hq, device="cuda"), echo.BlockAttentionWorkspace(4, D)
        t, ctx = dev(table), i32(lens)
        echo.echo_block_attention(echo.make_block_attention_args(q, rows, t, ctx, Hkv, D ** -0.5, out, lse, ws, fmt=fmt, block_tokens=bs))
        acc = torch.zeros(2, Hkv, table.shape[1] * bs, device="cuda")
        echo.echo_block_weights(echo.make_block_weights_args(q, rows, t, ctx, Hkv, D ** -0.5, lse, None, acc, fmt=fmt, block_tokens=bs))
        total = acc.double().sum(-1).cpu().numpy()
        # both sides' scores: (D + 4) 2^-23 of magnitudes below 60, twice
        assert np.abs(total - 4).max() <= 4 * (2 * (D + 4) * 2.0 ** -23 * 60 + 1e-5)


def test_weights_empty_rows_bad_ids_and_nonfinite_keys():
    g = np.random.default_rng(11)
    bs, D = 16, 64
    c = mr.Cache(BF16, bs, D, 1, 3, g)
    c.rows.view(np.uint16)[0, 4 * D + 7] = 0x7FC0              # token 4's key
    table = np.array([[0, 50, 2], [1, -1, -1]], np.int32)      # 50: outside
    q = torch.from_numpy(g.standard_normal((2, 1, 2, D)).astype(np.float32)).bfloat16().cuda()
    lse = torch.tensor([[[3.0, -np.inf]], [[-np.inf, -np.inf]]], device="cuda")
    out, st = torch.zeros(2, 1, 48, device="cuda"), status()
    echo.echo_block_weights(echo.make_block_weights_args(q, c.dev(), dev(table), i32([60, 10]), 1, 0.1, lse, None, out, block_tokens=bs,
                                                         dev_status=st))
    got = out.cpu().numpy()[:, 0]
    assert np.isnan(got[0, 4]) and np.isfinite(np.delete(got[0], 4)).all() and (got[0, 16:32] == 0).all()
    assert (np.delete(got[0, :16], 4) > 0).all() and (got[0, 32:] > 0).all()
    assert (got[1] == 0).all() and int(st) == echo.DEV_BAD_INDEX   # (a length of 60 in 48 slots, too)


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------

def run_evict(fmt, D, bs, Hkv, lens, keep, sinks=0, recent=0, new=None, acc=None, in_place=False, heads=False, seed=0, twice=True):
    g = np.random.default_rng(seed)
    B = len(lens)
    table, n = mr.tables(lens, bs, Hkv, g, heads=heads)
    c = mr.Cache(fmt, bs, D, Hkv, n if not heads else -(-n // Hkv), g)
    T = table.shape[-1] * bs
    if acc is None:
        acc = np.exp(g.standard_normal((B, Hkv, T))).astype(np.float32)
        acc[g.random(acc.shape) < 0.2] = 0
    known = np.maximum(0, np.array(lens) - (new if new is not None else max(lens)))
    nxt = np.array(lens) + np.where(known > 0, 50, 0)
    pos = np.full((B, Hkv, T), -9, np.int32)
    full = np.zeros((B, Hkv, T), np.int64)
    for b in range(B):
        for h in range(Hkv):
            pos[b, h, :known[b]] = g.permutation(nxt[b] - lens[b] + known[b])[:known[b]]
        full[b] = np.where(np.arange(T) < known[b], pos[b], nxt[b] - lens[b] + np.arange(T))
    rows, t, st = c.dev(), dev(table), status()
    a, p = torch.from_numpy(acc).cuda(), dev(pos)
    a_out = a if in_place else torch.full_like(a, 9.0)
    p_out = p if in_place else torch.full_like(p, 9)
    ln = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    kw = dict(pos=p, pos_out=p_out, pos_len=i32(known), next_pos=i32(nxt)) if recent or in_place or seed % 2 else {}
    args = echo.make_block_evict_args(rows, t, i32(lens), ln, Hkv, keep, a, a_out, echo.BlockEvictWorkspace(B, Hkv, keep), sinks=sinks,
                                      recent=recent, fmt=fmt, block_tokens=bs, dev_status=st, **kw)
    for _ in range(2 if twice and not in_place else 1):       # (a repeated call: the same again)
        echo.echo_block_evict(args)
    got, got_pos, got_rows = a_out.cpu().numpy(), p_out.cpu().numpy(), rows.cpu().numpy().view(np.uint8).reshape(c.rows.shape)
    want_rows = c.rows.copy()
    assert int(st) == 0 and ln.tolist() == [min(m, keep) for m in lens]
    for b, m in enumerate(lens):
        e = min(m, keep)
        for h in range(Hkv):
            src = mr.evict(acc[b, h].astype(np.float64), full[b, h], m, keep, sinks, recent, int(nxt[b]))
            assert np.array_equal(got[b, h, :e], acc[b, h, src], equal_nan=True), (b, h)
            if kw:
                assert (got_pos[b, h, :e] == full[b, h, src]).all()
            if not in_place:
                assert (got[b, h, e:] == 9.0).all()
            for d in np.nonzero(src != np.arange(len(src)))[0]:
                s = int(src[d])
                r0, r1 = mr.row_of(table, Hkv, b, h, s // bs), mr.row_of(table, Hkv, b, h, int(d) // bs)
                for x, y in zip(ref.token_bytes(fmt, bs, D, s % bs), ref.token_bytes(fmt, bs, D, int(d) % bs)):
                    want_rows[r1, y] = c.rows[r0, x]
    assert (got_rows == want_rows).all()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D,bs,Hkv", [(128, 64, 2), (64, 16, 3), (128, 48, 1), (64, 128, 2)])
def test_evict(fmt, D, bs, Hkv):
    run_evict(fmt, D, bs, Hkv, [0, 1, 40, 41, 100, 300], 40)
    run_evict(fmt, D, bs, Hkv, [33, 36, 200, 64], 32, sinks=4, recent=8, new=3, seed=1)
    run_evict(fmt, D, bs, Hkv, [90, 20], 1, seed=2, heads=True)
    run_evict(fmt, D, bs, Hkv, [150, 149], 140, sinks=2, recent=138, new=10, seed=3, in_place=True)


@pytest.mark.parametrize("kind", ["equal", "zeros", "wild", "heavy"])
def test_evict_ties_and_odd_weights(kind):
    g = np.random.default_rng(5)
    acc = np.exp(3 * g.standard_normal((2, 2, 320))).astype(np.float32)
    if kind == "equal":
        acc[:] = 0.125
    elif kind == "zeros":
        acc[g.random(acc.shape) < 0.9] = 0
    elif kind == "wild":
        pool = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, 3e38, -1.0], np.float32)
        acc = np.where(g.random(acc.shape) < 0.6, pool[g.integers(0, 8, acc.shape)], acc)
    else:
        acc[..., 7] = 1e30
    for keep in (1, 100, 250, 299):
        run_evict(BF16, 64, 32, 2, [300, 320], keep, sinks=min(1, keep), acc=acc.copy(), seed=7)


@pytest.mark.parametrize("lens,keep,recent", [([3000, 2500], 1000, 100), ([9000], 8000, 0), ([40000], 600, 64), ([20000], 16, 0)])
def test_evict_long(lens, keep, recent):
    """Both numbers of threads, moves in a kernel of their own, keys that shared memory does not hold."""
    run_evict(FP4, 64, 64, 1, lens, keep, sinks=2, recent=recent, seed=len(lens))


@pytest.mark.parametrize("slots", [8192, 8256, 10048, 10112, 10240, 12288, 32768, 32832])
def test_evict_at_the_edges_of_shared_memory(slots):
    """Contexts whose keys, beside what the kernel holds in any case, take just under and over 48 KB of it."""
    run_evict(BF16, 64, 64, 1, [slots], 300, sinks=4, recent=100, seed=9, twice=False)


def test_evict_runs_of_more_slots_than_marks():
    """More than 64 slots a thread."""
    run_evict(FP4, 64, 64, 1, [70000, 66001], 800, sinks=4, recent=64, new=100, seed=13, twice=False)
    acc = np.full((1, 1, 67008), 0.5, np.float32)
    run_evict(FP4, 64, 64, 1, [67000], 66000, acc=acc, seed=14, twice=False)


def test_evict_more_recent_positions_than_room():
    """Positions that repeat (a caller's mistake): more tokens are recent than may stay; the first slots do."""
    g = np.random.default_rng(8)
    table, n = mr.tables([40], 16, 1, g)
    c = mr.Cache(BF16, 16, 64, 1, n, g)
    acc, pos = torch.rand(1, 1, 48, device="cuda"), torch.full((1, 1, 48), 99, dtype=torch.int32, device="cuda")
    out, pout, ln = torch.zeros_like(acc), torch.zeros_like(pos), i32([0])
    echo.echo_block_evict(echo.make_block_evict_args(c.dev(), dev(table), i32([40]), ln, 1, 10, acc, out, echo.BlockEvictWorkspace(1, 1, 10),
                                                     recent=4, pos=pos, pos_out=pout, pos_len=i32([40]), next_pos=i32([100]),
                                                     block_tokens=16))
    assert (out[0, 0, :10] == acc[0, 0, :10]).all() and int(ln) == 10


def test_evict_bad_ids_move_nothing():
    g = np.random.default_rng(9)
    c = mr.Cache(BF16, 16, 64, 1, 4, g)
    table = np.array([[0, 99, -1, 3]], np.int32)
    acc = np.zeros((1, 1, 64), np.float32)
    acc[0, 0, 20], acc[0, 0, 40], acc[0, 0, 50] = 3, 2, 1       # in the bad block, in the missing one, and held
    rows, st, ln = c.dev(), status(), i32([0])
    out = torch.zeros(1, 1, 64, device="cuda")
    echo.echo_block_evict(echo.make_block_evict_args(rows, dev(table), i32([80]), ln, 1, 3, dev(acc), out, echo.BlockEvictWorkspace(1, 1, 3),
                                                     block_tokens=16, dev_status=st))
    want = c.rows.copy()
    for x, y in zip(ref.token_bytes(BF16, 16, 64, 50 % 16), ref.token_bytes(BF16, 16, 64, 2)):
        want[0, y] = c.rows[3, x]
    assert (rows.cpu().numpy().view(np.uint8).reshape(want.shape) == want).all()
    assert int(st) == echo.DEV_BAD_INDEX and int(ln) == 3 and out[0, 0, :3].tolist() == [3.0, 2.0, 1.0]


def test_binding_refuses():
    f, i = (lambda *s: torch.zeros(s, device="cuda")), (lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda"))
    rows = torch.zeros(4, echo.block_row_elems(BF16, 16, 64), dtype=torch.int16, device="cuda")
    ok = dict(rows=rows, table=i(1, 2), length=i(1), len_out=i(1), n_kv_heads=2, keep=4, acc=f(1, 2, 32), acc_out=f(1, 2, 32),
              ws=echo.BlockEvictWorkspace(1, 2, 4), block_tokens=16)
    echo.echo_block_evict(echo.make_block_evict_args(**ok))
    for bad in (dict(acc=f(1, 2, 31)), dict(acc_out=f(1, 1, 32)), dict(table=i(2, 2)), dict(pos=i(1, 2, 33)), dict(length=i(2)),
                dict(rows=rows[:, :100].contiguous()), dict(acc=f(1, 2, 32).double()), dict(len_out=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(echo.EchoError):
            echo.make_block_evict_args(**{**ok, **bad})
    small = echo.make_block_evict_args(**{**ok, "keep": 400})
    with pytest.raises(echo.EchoError, match="workspace"):
        echo.echo_block_evict(small)
