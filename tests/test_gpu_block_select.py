"""echo_block_summary (exact), echo_block_scores (64-bit bound within a derived tolerance) and
echo_block_select (exact) on the GPU."""
import numpy as np
import pytest
import torch

import block_ref as ref
import more_ref as mr
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev

pytestmark = pytest.mark.gpu
BF16, FP4 = echo.BLOCK_BF16, echo.BLOCK_FP4
bf16 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().cuda()
status = lambda: torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# summaries
# ---------------------------------------------------------------------------

def check_summary(fmt, D, bs, Hkv, lens, old, heads=False, gaps=0.0, k_shift=0, scale=1.0, seed=0):
    g = np.random.default_rng(seed)
    table, n = mr.tables(np.maximum(lens, old if old is not None else 0), bs, Hkv, g, heads=heads, gaps=gaps)
    c = mr.Cache(fmt, bs, D, Hkv, n if not heads else -(-n // Hkv), g, scale=scale * 2.0 ** k_shift)
    want = np.full((c.rows.shape[0], 2, D), 77.0)
    for b, m in enumerate(lens):
        o = 0 if old is None else old[b]
        if m == o:
            continue
        for i in range(min(m, o) // bs, -(-m // bs)):
            for h in range(Hkv):
                r = mr.row_of(table, Hkv, b, h, i)
                if r < 0:
                    continue
                e = min(bs, m - i * bs)
                c.spoil(r, range(e, bs))       # tokens past the length may hold any bytes
                k = c.k[r, :e] * 2.0 ** -k_shift
                want[r, 0], want[r, 1] = k.min(0), k.max(0)
    out = bf16(np.full(want.shape, 77.0))
    st = status()
    echo.echo_block_summary(echo.make_block_summary_args(
        c.dev(), dev(table), dev(np.array(lens, np.int32)), Hkv, out, old_len=None if old is None else dev(np.array(old, np.int32)),
        fmt=fmt, block_tokens=bs, k_shift=k_shift, dev_status=st))
    assert (out.double().cpu().numpy() == want).all() and int(st) == 0


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D,bs,Hkv", [(128, 64, 2), (64, 16, 3), (128, 48, 1), (64, 128, 2), (128, 16, 8)])
def test_summary(fmt, D, bs, Hkv):
    check_summary(fmt, D, bs, Hkv, [0, 1, bs - 1, bs, bs + 1, 3 * bs + 5, 7], None)
    check_summary(fmt, D, bs, Hkv, [5, bs, bs + 1, 2 * bs, 2 * bs, 0, 3 * bs], [4, bs - 1, bs, 2 * bs, bs + 1, 9, 0], heads=True, seed=1)
    # tokens taken back: the block that holds the last one is summed up anew
    check_summary(fmt, D, bs, Hkv, [bs, bs + 1, 1, 2 * bs - 1], [bs + 3, 2 * bs, bs, 3 * bs], gaps=0.2, seed=2)


def test_summary_of_many_requests_and_shifts():
    check_summary(BF16, 64, 16, 2, list(np.random.default_rng(0).integers(0, 70, 300)), None, seed=3)
    check_summary(FP4, 128, 32, 2, [40, 64, 1], None, k_shift=7, scale=2.0 ** -7, seed=4)
    check_summary(FP4, 64, 32, 2, [40, 64, 1], None, k_shift=-5, scale=32.0, seed=5)


def test_summary_more_requests_than_shared_memory_holds_at_first():
    lens = np.zeros(16384, np.int64)
    lens[[0, 77, 12000, 16383]] = [3, 20, 16, 33]
    check_summary(BF16, 64, 16, 1, list(lens), None, seed=6)


def test_summary_nan_keys_and_bad_ids():
    g = np.random.default_rng(7)
    c = mr.Cache(BF16, 16, 64, 2, 4, g)
    c.rows.view(np.uint16)[2, 5 * 64 + 9] = 0x7FC0           # block 1, head 0: token 5, dim 9
    table = np.array([[1, 9, -1, 3]], np.int32)               # 9: outside the 4 blocks
    out = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    st = status()
    echo.echo_block_summary(echo.make_block_summary_args(c.dev(), dev(table), dev(np.array([100], np.int32)), 2, out, block_tokens=16,
                                                         dev_status=st))
    got = out.double().cpu().numpy()
    assert np.isnan(got[2, :, 9]).all() and np.isfinite(np.delete(got[2], 9, 1)).all()
    assert (got[[0, 1, 4, 5]] == 0).all() and int(st) == echo.DEV_BAD_INDEX       # and the length is above 64
    assert (got[7, 0] == c.k[7].min(0)).all() and (got[7, 1] == c.k[7].max(0)).all()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D,bs", [(128, 128), (64, 256), (128, 208)])
def test_summary_of_large_blocks(fmt, D, bs):
    check_summary(fmt, D, bs, 2, [0, 1, bs - 1, bs, bs + 1, 3 * bs + 5, 7], None, seed=7)
    check_summary(fmt, D, bs, 2, [5, bs, bs + 60, 2 * bs, 2 * bs, 0], [4, bs - 1, bs, 2 * bs, bs + 1, 9], gaps=0.2, seed=8)


# ---------------------------------------------------------------------------
# scores
# ---------------------------------------------------------------------------

def check_scores(D, bs, Hq, Hkv, n_q, lens, scale=None, heads=False, gaps=0.0, seed=0):
    g = np.random.default_rng(seed)
    B, G = len(lens), Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    table, n = mr.tables(lens, bs, Hkv, g, heads=heads, gaps=gaps)
    rows = n if heads else n * Hkv
    mid, half = g.standard_normal((rows, D)), np.abs(g.standard_normal((rows, D)))
    lo, hi = ref.bf16_round(mid - half), ref.bf16_round(mid + half)
    q = ref.bf16_round(g.standard_normal((B, n_q, Hq, D)))
    out = torch.full((B, n_q, Hkv, table.shape[-1]), 1234.0, device="cuda")
    st = status()
    echo.echo_block_scores(echo.make_block_scores_args(bf16(q), bf16(np.stack([lo, hi], 1)), dev(table), dev(np.array(lens, np.int32)),
                                                       Hkv, scale, out, block_tokens=bs, dev_status=st))
    got = out.double().cpu().numpy()
    assert int(st) == 0
    for b in range(B):
        for j in range(n_q):
            nb = -(-max(0, lens[b] - (n_q - 1 - j)) // bs)
            assert (got[b, j, :, nb:] == 1234.0).all()        # left as they were
            for h in range(Hkv):
                for i in range(nb):
                    r = mr.row_of(table, Hkv, b, h, i)
                    if r < 0:
                        assert got[b, j, h, i] == -np.inf
                        continue
                    x = q[b, j, h * G:(h + 1) * G] * scale
                    p = np.maximum(x * lo[r], x * hi[r])
                    # 2 D products (half of them zeros) summed in fp32, each addition off by 2^-23 of the
                    # magnitudes' sum at most (the tensor cores cut off), and one product with the scale
                    mag = np.maximum(np.abs(x * lo[r]), np.abs(x * hi[r])).sum(-1).max()
                    want = p.sum(-1).max()
                    assert abs(got[b, j, h, i] - want) <= (2 * D + 2) * 2.0 ** -23 * mag + 1e-30, (b, j, h, i)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n_q", [(8, 1, 1), (2, 2, 5), (8, 4, 3), (6, 2, 2), (16, 4, 1), (10, 2, 4), (16, 1, 2), (24, 1, 3), (80, 1, 2),
                                        (3, 3, 17)])
def test_scores(D, Hq, Hkv, n_q):
    check_scores(D, 16, Hq, Hkv, n_q, [0, 1, 2, 16, 17, 16 * 15 + 3, 16 * 40], gaps=0.1)


def test_scores_of_long_contexts_tables_per_head_and_scales():
    check_scores(128, 64, 16, 2, 1, [64 * 700 + 1, 64 * 300], heads=True, seed=1)
    check_scores(64, 48, 8, 4, 2, [48 * 70, 5], scale=-0.3, seed=2)
    check_scores(64, 32, 4, 2, 1, [100], scale=0.0, seed=3)


@pytest.mark.parametrize("D,Hq,Hkv,n_q", [(64, 8, 2, 150), (128, 12, 4, 70), (64, 32, 2, 40), (64, 2, 2, 300), (64, 70, 1, 5)])
def test_scores_of_many_query_tokens(D, Hq, Hkv, n_q):
    """Columns that are split over CTAs, of groups that fill a chunk and of those that do not."""
    check_scores(D, 16, Hq, Hkv, n_q, [n_q, n_q - 3, 16 * 9 + 5], gaps=0.1, seed=n_q)


def test_scores_bound_the_keys():
    """Every key's score is below its block's, up to the rounding of both."""
    g = np.random.default_rng(4)
    D, bs, Hq, Hkv, lens = 128, 32, 8, 2, [150, 64]
    for fmt in (BF16, FP4):
        table, n = mr.tables(lens, bs, Hkv, g)
        c = mr.Cache(fmt, bs, D, Hkv, n, g)
        q = ref.bf16_round(g.standard_normal((2, 1, Hq, D)))
        rows, t, ctx = c.dev(), dev(table), dev(np.array(lens, np.int32))
        summary = torch.zeros(rows.shape[0], 2, D, dtype=torch.bfloat16, device="cuda")
        scores = torch.zeros(2, 1, Hkv, table.shape[1], device="cuda")
        echo.echo_block_summary(echo.make_block_summary_args(rows, t, ctx, Hkv, summary, fmt=fmt, block_tokens=bs))
        echo.echo_block_scores(echo.make_block_scores_args(bf16(q), summary, t, ctx, Hkv, 1.0, scores, block_tokens=bs))
        got = scores.double().cpu().numpy()
        for b in range(2):
            for h in range(Hkv):
                k = mr.tokens_of(c, table, b, h, lens[b])[0]
                x = (k @ q[b, 0, h * 4:h * 4 + 4].T).max(1)
                mag = (np.abs(k) @ np.abs(q[b, 0, h * 4:h * 4 + 4]).T).max()
                for i in range(-(-lens[b] // bs)):
                    assert got[b, 0, h, i] >= x[i * bs:(i + 1) * bs].max() - 4 * D * 2.0 ** -23 * mag


def test_scores_bad_ids_and_lengths():
    g = np.random.default_rng(5)
    table = np.array([[0, 7, -1]], np.int32)
    s = bf16(g.standard_normal((4, 2, 64)))
    out, st = torch.zeros(1, 1, 2, 3, device="cuda"), status()
    echo.echo_block_scores(echo.make_block_scores_args(bf16(g.standard_normal((1, 1, 4, 64))), s, dev(table), dev(np.array([500], np.int32)),
                                                       2, 0.1, out, block_tokens=16, dev_status=st))
    got = out.cpu().numpy()
    assert np.isfinite(got[..., 0]).all() and (got[..., 1:] == -np.inf).all() and int(st) == echo.DEV_BAD_INDEX


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------

def check_select(scores, lens, bs, k, first=0, last=0, table=None, seed=0):
    B, n_q, Hkv, n = scores.shape
    e = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
    sel, rows, ln = e(B, n_q, Hkv, k), e(B, n_q, Hkv, k) if table is not None else None, e(B, n_q)
    st = status()
    echo.echo_block_select(echo.make_block_select_args(torch.from_numpy(scores).cuda(), dev(np.array(lens, np.int32)), sel, block_tokens=bs,
                                                       first=first, last=last, table=dev(table) if table is not None else None,
                                                       sel_rows=rows, len_out=ln, dev_status=st))
    got, got_rows = sel.cpu().numpy(), rows.cpu().numpy() if rows is not None else None
    assert int(st) == 0
    for b in range(B):
        for j in range(n_q):
            m = max(0, lens[b] - (n_q - 1 - j))
            assert int(ln[b, j]) == m
            nb = -(-m // bs)
            for h in range(Hkv):
                held = [table is None or mr.row_of(table, Hkv, b, h, i) >= 0 for i in range(nb)]
                want = mr.select(scores[b, j, h].astype(np.float64), nb, k, first, last, held)
                assert list(got[b, j, h]) == want, (b, j, h)
                if rows is not None:
                    assert list(got_rows[b, j, h]) == [mr.row_of(table, Hkv, b, h, i) if i >= 0 else -1 for i in want]


@pytest.mark.parametrize("n", [1, 7, 32, 33, 100, 256, 257, 700, 1024])
@pytest.mark.parametrize("kind", ["random", "coarse", "equal", "wild"])
def test_select(n, kind):
    g = np.random.default_rng(n)
    B, n_q, Hkv, bs = 3, 2, 2, 16
    x = g.standard_normal((B, n_q, Hkv, n)).astype(np.float32)
    if kind == "coarse":
        x = np.round(x * 2) / 2
    elif kind == "equal":
        x[:] = -0.25
    elif kind == "wild":                # infinities, NaN, both zeros, denormals, huge and tiny ones
        pool = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-42, -1e-42, 3e38, -3e38, 1.0, 1e-30], np.float32)
        x = np.where(g.random(x.shape) < 0.7, pool[g.integers(0, len(pool), x.shape)], x * 1e20).astype(np.float32)
    lens = [n * bs, max(0, n * bs - 20), min(n * bs, 5)]
    for k, first, last in [(1, 0, 0), (4, 1, 2), (16, 0, 1), (40, 40, 0), (n + 3, 1, 1), (3, 0, 3)]:
        check_select(x, lens, bs, k, first, last if first + last <= k else 0)


def test_select_held_blocks_only_and_empty_contexts():
    g = np.random.default_rng(1)
    for heads in (False, True):
        lens = [16 * 60, 0, 1, 333]
        table, _ = mr.tables(lens, 16, 3, g, heads=heads, gaps=0.5)
        x = np.round(g.standard_normal((4, 3, 3, table.shape[-1])) * 4).astype(np.float32)
        check_select(x, lens, 16, 9, 1, 2, table=table)
        check_select(x, lens, 16, 64, 0, 0, table=table)


@pytest.mark.parametrize("B,n_q,Hkv,n,k", [(1, 800, 2, 1000, 8), (2, 1, 2, 4096, 32), (1, 3, 1, 20000, 17), (1, 1, 1, 32768, 128),
                                           (700, 1, 1, 40, 5), (1, 2, 1, 1025, 500)])
def test_select_sizes(B, n_q, Hkv, n, k):
    g = np.random.default_rng(n)
    x = g.standard_normal((B, n_q, Hkv, n)).astype(np.float32)
    x[..., ::3] = np.round(x[..., ::3] * 3) / 3
    check_select(x, [max(n_q, n * 32 - 40 * b) for b in range(B)], 32, k, 1, 1)


@pytest.mark.parametrize("rows", [2, 800])
@pytest.mark.parametrize("n", [256, 509, 512, 1022, 1500, 2048, 3001, 4096, 6000, 8192, 12345, 16384, 30000])
def test_select_every_width(rows, n):
    """All numbers of warps and of blocks per thread, rows that start on 16-byte boundaries and not."""
    g = np.random.default_rng(rows + n)
    x = g.standard_normal((1, rows, 1, n)).astype(np.float32)
    x[0, 0, 0, 5::7] = np.inf
    x[0, 1, 0] = np.round(x[0, 1, 0] * 2) / 2
    check_select(x[:, :min(rows, max(2, 1300000 // n))], [n * 16 - 3], 16, 37, 1, 2)


def test_select_length_above_the_table():
    x = np.arange(8, dtype=np.float32).reshape(1, 1, 1, 8)
    sel, ln, st = (torch.zeros(1, 1, 1, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), status())
    echo.echo_block_select(echo.make_block_select_args(torch.from_numpy(x).cuda(), dev(np.array([1000], np.int32)), sel, block_tokens=16,
                                                       len_out=ln, dev_status=st))
    assert sel.flatten().tolist() == [6, 7] and int(ln) == 128 and int(st) == echo.DEV_BAD_INDEX


def test_binding_refuses():
    x, i = torch.zeros(1, 1, 2, 8, device="cuda"), lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    ok = dict(scores=x, ctx_len=i(1), sel=i(1, 1, 2, 2), block_tokens=16)
    echo.echo_block_select(echo.make_block_select_args(**ok))
    for bad in (dict(scores=x.double()), dict(scores=x.cpu()), dict(sel=i(1, 1, 3, 2)), dict(ctx_len=i(2)), dict(table=i(1, 7)),
                dict(sel_rows=i(1, 1, 2, 3), table=i(1, 8)), dict(len_out=i(1)), dict(scores=x.transpose(2, 3))):
        with pytest.raises(echo.EchoError):
            echo.make_block_select_args(**{**ok, **bad})
    with pytest.raises(echo.EchoError):
        echo.make_block_summary_args(torch.zeros(4, 100, dtype=torch.int16, device="cuda"), i(1, 2), i(1), 2,
                                     torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda"), block_tokens=16)
