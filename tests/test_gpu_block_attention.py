"""echo_block_attention on the GPU against a 64-bit softmax over the tokens each query sees,
within bounds derived from the arithmetic (block_ref.attention_bounds).  Bytes of tokens no
query sees are NaN patterns throughout."""
import numpy as np
import pytest
import torch

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev

pytestmark = pytest.mark.gpu
BF16, FP4 = echo.BLOCK_BF16, echo.BLOCK_FP4


class Attn:
    def __init__(self, fmt, D, bs, Hq, Hkv, n_q, lens, sinks=0, window=0, heads=False, sel=None, seed=0, qscale=1.0,
                 spare=3, cap=None):
        g = np.random.default_rng(seed)
        self.__dict__.update(fmt=fmt, D=D, bs=bs, Hq=Hq, Hkv=Hkv, n_q=n_q, lens=np.array(lens, np.int32), sinks=sinks,
                             window=window, G=Hq // Hkv, B=len(lens))
        self.scale = D ** -0.5
        self.q_np = ref.bf16_round(g.standard_normal((self.B, n_q, Hq, D)) * qscale)
        nblk = max(1, -(-max(max(lens), 1) // bs)) if cap is None else cap
        B = self.B
        if sel:          # entries: block index or -1, per (request, KV head)
            nblk_list = max(1, -(-max(max(lens), 1) // bs))
            self.sel = np.full((B, Hkv, sel), -1, np.int32)
            for b in range(B):
                for h in range(Hkv):
                    n = min(sel, nblk_list, -(-int(lens[b]) // bs))
                    pick = np.sort(g.permutation(-(-int(lens[b]) // bs))[:n]) if lens[b] > 0 else []
                    self.sel[b, h, :n] = pick
            ids = g.permutation(B * Hkv * sel + spare)[:B * Hkv * sel].reshape(B, Hkv, sel).astype(np.int32)
            self.table = np.where(self.sel >= 0, ids, -1).astype(np.int32)
            n_rows = B * Hkv * sel + spare
            self.logical = self.sel
        else:
            self.sel = None
            held = np.arange(nblk)[None] * bs < self.lens[:, None]
            if window:
                wlo = self.lens - (n_q - 1) - window
                at = np.arange(nblk)[None] * bs
                held &= (at < sinks) | (at + bs > wlo[:, None])
            if heads:
                ids = g.permutation(B * Hkv * nblk + spare)[:B * Hkv * nblk].reshape(B, Hkv, nblk).astype(np.int32)
                self.table = np.where(held[:, None], ids, -1).astype(np.int32)
                n_rows = B * Hkv * nblk + spare
            else:
                self.table = np.full((B, nblk), -1, np.int32)
                self.table[held] = g.permutation(int(held.sum()) + spare)[:int(held.sum())]
                n_rows = (int(held.sum()) + spare) * Hkv
            self.logical = np.broadcast_to(np.arange(nblk), (B, Hkv, nblk))
        R = echo.block_row_elems(fmt, bs, D)
        self.rows_np = np.full((n_rows, 2 * R), 0xFF, np.uint8)      # NaN in bf16, NaN scales in 4 bits
        self.kv = {}
        for b in range(B):
            for h in range(Hkv):
                for i in np.nonzero((self.table[b, h] if self.table.ndim == 3 else self.table[b]) >= 0)[0]:
                    row, lb = self.row(b, h, i), int(self.logical[b, h, i])
                    for off in range(bs):
                        p = lb * bs + off
                        if self.seen_by_some(b, p) and (row, off) not in self.kv:
                            k = ref.bf16_round(g.standard_normal(D))
                            v = ref.bf16_round(g.standard_normal(D))
                            self.kv[row, off] = ref.write_token(self.rows_np[row], fmt, bs, D, off, k, v)
        self.dev()

    def row(self, b, h, i):
        if self.table.ndim == 3:
            return int(self.table[b, h, i])
        t = int(self.table[b, i])
        return t * self.Hkv + h if t >= 0 else -1

    def sees(self, b, j, p):
        n = int(self.lens[b]) - (self.n_q - 1 - j)
        return p < n and (self.window == 0 or p >= n - self.window or p < self.sinks)

    def seen_by_some(self, b, p):
        n = int(self.lens[b])
        return p < n and (self.window == 0 or p >= n - (self.n_q - 1) - self.window or p < self.sinks)

    def dev(self, rows=None):
        bf = lambda x: dev(ref.bf16_bits(x).view(np.int16).reshape(x.shape)).view(torch.bfloat16)
        self.q, self.rows = bf(self.q_np), dev(self.rows_np.view(np.int16))
        self.t, self.s = dev(self.table), None if self.sel is None else dev(self.sel)
        self.ctx = dev(self.lens)
        self.out = torch.full((self.B, self.n_q, self.Hq, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.B, self.n_q, self.Hq), float("nan"), device="cuda")
        self.ws = echo.BlockAttentionWorkspace(self.n_q * self.G, self.D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self, **kw):
        a = dict(rows=self.rows, ws=self.ws, table=self.t, lse=self.lse, out=self.out)
        a.update(kw)
        return echo.make_block_attention_args(self.q, a["rows"], a["table"], self.ctx, self.Hkv, self.scale, a["out"],
                                              a["lse"], a["ws"], fmt=self.fmt, block_tokens=self.bs, sel=self.s,
                                              sinks=self.sinks, window=self.window, dev_status=self.status)

    def want(self):
        shape = (self.B, self.n_q, self.Hq)
        out, av, sv = (np.zeros(shape + (self.D,)) for _ in range(3))
        lse, mag, tiny, n = np.full(shape, -np.inf), np.zeros(shape), np.zeros(shape), np.zeros(shape)
        for b in range(self.B):
            for h in range(self.Hkv):
                tok = []                                    # (position, k, v), entry after entry
                for i in np.nonzero((self.table[b, h] if self.table.ndim == 3 else self.table[b]) >= 0)[0]:
                    row, lb = self.row(b, h, i), int(self.logical[b, h, i])
                    if 0 <= row < self.rows_np.shape[0] and lb >= 0:
                        tok += [(lb * self.bs + o, *self.kv[row, o]) for o in range(self.bs) if (row, o) in self.kv]
                hs = slice(h * self.G, (h + 1) * self.G)
                for j in range(self.n_q):
                    mine = [(k, v) for p, k, v in tok if self.sees(b, j, p)]
                    if not mine:
                        continue
                    k, v = np.array([m[0] for m in mine]), np.array([m[1] for m in mine])
                    r = ref.attention(self.q_np[b, j, hs], [(k, v)] * self.G, self.scale)
                    out[b, j, hs], lse[b, j, hs], av[b, j, hs], mag[b, j, hs], tiny[b, j, hs], sv[b, j, hs] = r
                    n[b, j, hs] = len(mine)
        return n, (out, lse, av, mag, tiny, sv)

    def check(self, status=0):
        torch.cuda.synchronize()
        n, want = self.want()
        out, lse = want[:2]
        far, far_lse = ref.attention_bounds(self.fmt, self.D, n, *want)
        got, got_lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        assert int(self.status) == status
        assert np.isfinite(got).all()
        assert (np.abs(got - out) <= far).all(), (np.abs(got - out) / np.maximum(far, 1e-30)).max()
        live = np.isfinite(lse)
        assert np.array_equal(np.isfinite(got_lse), live) and (got_lse[~live] == -np.inf).all()
        assert (np.abs(got_lse[live] - lse[live]) <= far_lse[live]).all()


FORMATS = [(BF16, 128), (FP4, 128), (BF16, 64), (FP4, 64)]
# Blocks of the table beyond the contexts: tables that may hold long contexts take the path
# that cuts all contexts into equal pieces and merges them in a second kernel, others a CTA
# or a cluster per (request, KV head).
WIDE = 60000


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens", [[0], [1], [0, 1, 2], [15, 16, 17, 31, 32, 33], [63, 64, 65, 0, 127, 128, 129, 200],
                                  [700, 3, 0, 1025, 64, 0]])
def test_lengths(fmt, D, lens, wide):
    a = Attn(fmt, D, 64, 8, 2, 1, lens, seed=len(lens), cap=WIDE // 64 if wide else None)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,n_q", [(1, 1, 1), (3, 1, 1), (7, 1, 2), (16, 1, 1), (12, 4, 3), (20, 2, 3), (33, 1, 1),
                                        (8, 8, 4), (64, 8, 5), (48, 1, 2)])
@pytest.mark.parametrize("wide", [False, True])
def test_groups_and_query_tokens(fmt, D, Hq, Hkv, n_q, wide):
    a = Attn(fmt, D, 32, Hq, Hkv, n_q, [330, 5, 1, 77], seed=Hq, cap=WIDE // 32 if wide else None)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,n_q", [(17, 1, 1), (10, 2, 4), (24, 2, 2), (25, 1, 1), (56, 1, 1), (3, 1, 19)])
@pytest.mark.parametrize("wide", [False, True])
def test_rows_that_fill_three_columns_and_one_more(fmt, D, Hq, Hkv, n_q, wide):
    a = Attn(fmt, D, 32, Hq, Hkv, n_q, [1300, 17, 0, 33], sinks=3, window=400, seed=Hq, cap=WIDE // 32 if wide else None)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("bs", [16, 48, 128, 256])
@pytest.mark.parametrize("heads", [False, True])
def test_block_sizes_and_tables_per_head(fmt, bs, heads):
    a = Attn(fmt, 128, bs, 8, 4, 1, [300, 1, 49, 128], heads=heads, seed=bs)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("sinks,window", [(0, 1), (0, 64), (4, 100), (4, 1), (16, 16), (65, 130), (1000, 5), (3, 2000)])
def test_window_and_sinks(fmt, D, sinks, window):
    a = Attn(fmt, D, 32, 8, 2, 2, [700, 0, 1, 2, 90, 33], sinks=sinks, window=window, seed=window)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt,D", FORMATS)
def test_a_long_window_over_cut_contexts(fmt, D):
    a = Attn(fmt, D, 64, 4, 1, 2, [2600, 0, 700, 1], sinks=70, window=1800, seed=5)
    b = Attn(fmt, D, 64, 4, 1, 2, [2600, 0, 700, 1], sinks=70, window=50000, seed=6, cap=WIDE // 64)
    for x in (a, b):
        echo.echo_block_attention(x.args())
        x.check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("k,bs,window", [(1, 64, 0), (5, 64, 0), (16, 16, 0), (9, 32, 40), (600, 64, 0)])
def test_recalled_selections(fmt, k, bs, window):
    a = Attn(fmt, 128, bs, 8, 2, 2, [500, 1, 0, 130], sel=k, window=window, sinks=4 if window else 0, seed=k)
    echo.echo_block_attention(a.args())
    a.check()


def test_a_block_listed_twice_counts_twice():
    a = Attn(BF16, 128, 16, 4, 1, 1, [64], sel=3, seed=4)
    a.sel[0, 0], a.table[0, 0] = [1, 1, 2], [a.table[0, 0, 1]] * 2 + [a.table[0, 0, 2]]
    for off in range(16):                                      # rows follow their (new) blocks
        for row in set(a.table[0, 0].tolist()):
            g = np.random.default_rng(row * 100 + off)
            a.kv[row, off] = ref.write_token(a.rows_np[row], BF16, 16, 128, off, ref.bf16_round(g.standard_normal(128)),
                                             ref.bf16_round(g.standard_normal(128)))
    a.dev()
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_blocks_that_are_not_held(fmt):
    """Entries of -1 are skipped silently, entries past the rows are skipped and flagged."""
    a = Attn(fmt, 128, 16, 4, 2, 1, [100, 200], seed=8)
    a.table[0, 2], a.table[1, [0, 5, 12]] = -1, -1
    a.dev()
    echo.echo_block_attention(a.args())
    a.check()
    a.table[1, 3] = 1 << 29
    a.dev()
    echo.echo_block_attention(a.args())
    a.check(echo.DEV_BAD_INDEX)
    a.table[:] = -1                                             # nothing held at all
    a.dev()
    echo.echo_block_attention(a.args())
    a.check()


def test_context_past_the_table_is_clamped_and_flagged():
    for cap in (3, 40):
        a = Attn(BF16, 128, 16, 4, 2, 1, [cap * 16, 20], seed=9, cap=cap)
        a.ctx.copy_(dev(np.array([cap * 16 + 5, 20], np.int32)))
        echo.echo_block_attention(a.args())
        a.check(echo.DEV_BAD_INDEX)
        a.ctx.copy_(dev(np.array([-7, -1], np.int32)))          # negative: empty
        a.lens[:] = 0
        a.status.zero_()
        echo.echo_block_attention(a.args())
        a.check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("qscale", [1e-30, 1e-4, 30.0])
def test_query_magnitudes(fmt, qscale):
    a = Attn(fmt, 128, 64, 8, 2, 1, [400, 65], qscale=qscale, seed=10)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(fmt, scale):
    a = Attn(fmt, 128, 64, 8, 2, 2, [400, 65, 0], seed=11, sinks=2, window=90)
    a.scale = scale
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_a_growing_maximum_rescales_what_came_before(fmt):
    """Scores that climb by 300 over the context (and one late peak) move the running
    maximum many times; early tokens end up far below."""
    a = Attn(fmt, 64, 16, 4, 1, 1, [600], seed=12)
    a.q_np[:] = 1.0
    for i in range(38):
        row = a.row(0, 0, i)
        for off in range(16):
            p = i * 16 + off
            if p < 600:
                k = np.full(64, ref.bf16_round(np.array(p * 0.0625)))
                v = ref.bf16_round(np.random.default_rng(p).standard_normal(64))
                a.kv[row, off] = ref.write_token(a.rows_np[row], fmt, 16, 64, off, k, v)
    a.dev()
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("cap", [None, WIDE // 64])
@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_a_long_ragged_batch(fmt, cap):
    """Contexts split over many CTAs beside short and empty ones."""
    a = Attn(fmt, 128, 64, 8, 1, 1, [9000, 0, 17, 3000, 1, 64], seed=13, cap=cap)
    echo.echo_block_attention(a.args())
    a.check()
    first = a.out.clone(), a.lse.clone()
    for _ in range(3):                                          # the same bits every time
        echo.echo_block_attention(a.args())
        torch.cuda.synchronize()
        assert torch.equal(a.out, first[0]) and torch.equal(a.lse, first[1])


def test_no_lse_and_many_requests():
    a = Attn(BF16, 64, 16, 2, 1, 1, [int(x) for x in np.random.default_rng(3).integers(0, 60, 700)], seed=14)
    want = a.lse
    echo.echo_block_attention(a.args(lse=None))
    a.lse = torch.from_numpy(a.want()[1][1]).float().cuda()        # only the outputs are checked
    a.check()
    assert bool(torch.isnan(want).all())


def test_rows_past_4_gib():
    a = Attn(BF16, 128, 64, 8, 2, 1, [500, 200], seed=15)
    n = 5 * (1 << 30) // (4 * 64 * 128)
    big = torch.empty(n, 2 * 64 * 128, dtype=torch.int16, device="cuda")
    tail = a.rows.shape[0]
    assert n % 2 == 0 and tail % 2 == 0
    big[-tail:].copy_(a.rows)
    t = torch.where(a.t >= 0, a.t + (n - tail) // 2, -1).to(torch.int32)
    echo.echo_block_attention(a.args(rows=big, table=t))
    a.check()


@pytest.mark.parametrize("cap", [None, WIDE // 64])
def test_captured_graphs_share_a_workspace_in_turn(cap):
    """Two captured calls of different shapes with one workspace, replayed one after another
    on a side stream, with the lengths changed between replays."""
    x = Attn(BF16, 128, 64, 8, 1, 1, [3000, 40], seed=16, cap=cap)
    y = Attn(FP4, 128, 64, 8, 1, 1, [2500, 0, 900], seed=17, cap=cap)
    y.ws = x.ws
    st = torch.cuda.Stream()
    graphs = []
    for a in (x, y):
        echo.echo_block_attention(a.args())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            echo.echo_block_attention(a.args())
        graphs.append(g)
    for lens in ([3000, 40], [1, 33], [2999, 0], [0, 39]):      # (never past what the cache holds)
        x.lens[:] = lens
        x.ctx.copy_(dev(x.lens))
        x.out.fill_(float("nan")), y.out.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for g in graphs:
                g.replay()
        x.check(), y.check()


def test_two_streams_with_a_workspace_each():
    """Calls in flight at once on two streams, each with its own workspace."""
    a = [Attn(f, 128, 64, 8, 1, 1, [2000, 30, 700], seed=18 + i, cap=c)
         for i, (f, c) in enumerate(((BF16, WIDE // 64), (FP4, WIDE // 64), (BF16, None), (FP4, None)))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, x in enumerate(a):
            with torch.cuda.stream(streams[i % 2]):
                echo.echo_block_attention(x.args())
    for x in a:
        x.check()


@pytest.mark.parametrize("cap", [None, WIDE // 16])
def test_thousands_of_requests(cap):
    lens = np.zeros(5000, int)
    lens[[0, 17, 18, 2500, 4998, 4999]] = [5, 100, 33, 64, 1, 40]
    a = Attn(FP4, 64, 16, 2, 1, 1, [int(x) for x in lens], seed=22, cap=cap)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("Hq,n_q,window", [(8, 1, 0), (8, 2, 0), (3, 5, 40), (8, 3, 0)])
def test_many_short_requests(fmt, D, Hq, n_q, window):
    """More (request, KV head) pairs than SMs: two CTAs to an SM where the rows allow it."""
    lens = [int(x) for x in np.random.default_rng(Hq + n_q).integers(0, 130, 190)]
    a = Attn(fmt, D, 16, Hq, 1, n_q, lens, sinks=3 if window else 0, window=window, seed=23)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("D", [64, 128])
def test_many_contexts_cut_with_two_ctas_an_sm(D):
    """More pairs than SMs whose tables may hold 16384 tokens each: 4-bit rows, cut into twice
    as many pieces as SMs."""
    lens = [int(x) for x in np.random.default_rng(31).integers(0, 200, 160)]
    lens[7], lens[100] = 2100, 0
    a = Attn(FP4, D, 16, 8, 1, 1, lens, seed=32, cap=16384 // 16)
    echo.echo_block_attention(a.args())
    a.check()


def test_refused_workspaces_and_outputs():
    a = Attn(BF16, 128, 64, 8, 2, 1, [3])
    with pytest.raises(echo.EchoError, match="workspace"):
        a.args(ws=echo.BlockAttentionWorkspace(4, 128, device="cpu"))
    with pytest.raises(echo.EchoError, match="smaller"):
        echo.echo_block_attention(echo.make_block_attention_args(
            a.q.repeat(1, 4, 1, 1), a.rows, a.t, a.ctx, 2, 0.1, a.out.repeat(1, 4, 1, 1), None, a.ws))
    with pytest.raises(echo.EchoError, match="out must not"):
        echo.echo_block_attention(a.args(out=a.q))
