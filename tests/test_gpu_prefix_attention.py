"""echo_prefix_attention on the GPU against a 64-bit softmax over a request's prefix and its own
tokens, within bounds derived from the arithmetic.  Bytes of tokens no query sees are NaN patterns."""
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


class Shared:
    """Groups of requests behind prefixes `plens`, `start` the groups' first requests, own tokens
    `lens` (None: no own tokens at all)."""

    def __init__(self, fmt, D, bs, Hq, Hkv, n_q, plens, start, lens, B=None, heads=False, pheads=False, pgaps=0.0, gaps=0.0, scale=None,
                 k_shift=0, v_shift=0, qscale=1.0, seed=0):
        g = np.random.default_rng(seed)
        self.__dict__.update(fmt=fmt, D=D, bs=bs, Hq=Hq, Hkv=Hkv, n_q=n_q, plens=list(plens), start=list(start), G=Hq // Hkv,
                             k_shift=k_shift, v_shift=v_shift)
        self.B = B or len(lens)
        self.lens = list(lens) if lens is not None else None
        self.scale = D ** -0.5 if scale is None else scale
        self.q = ref.bf16_round(g.standard_normal((self.B, n_q, Hq, D)) * qscale)
        self.ptab, n0 = mr.tables(plens, bs, Hkv, g, heads=pheads, gaps=pgaps)
        blocks = -(-n0 // Hkv) if pheads else n0
        self.table, n1 = mr.tables(lens, bs, Hkv, g, heads=heads, gaps=gaps) if lens is not None else (None, 0)
        if lens is not None:     # the own rows lie behind the prefixes'
            self.table = np.where(self.table >= 0, self.table + blocks * (Hkv if heads else 1), -1).astype(np.int32)
        self.c = mr.Cache(fmt, bs, D, Hkv, blocks + (-(-n1 // Hkv) if heads else n1), g)
        for tab, ls in ((self.ptab, plens), (self.table, lens)):
            for b, m in enumerate(ls or []):
                for h in range(Hkv):
                    for i in range(m // bs, tab.shape[-1]):
                        r = mr.row_of(tab, Hkv, b, h, i)
                        if r >= 0:
                            self.c.spoil(r, range(max(0, m - i * bs), bs))

    def group(self, b):
        for g in range(len(self.plens)):
            if self.start[g] <= b < self.start[g + 1]:
                return g
        return None

    def args(self, q=None, ws=None, out=None, lse=True, stat=True):
        bf = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().cuda()
        self.qd = bf(self.q) if q is None else q
        self.out = torch.full_like(self.qd, 7.0) if out is None else out
        self.lse = torch.full(self.qd.shape[:3], 7.0, device="cuda") if lse else None
        self.ws = ws or echo.PrefixAttentionWorkspace(self.B, self.n_q, self.Hq, self.Hkv, self.D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.rows = self.c.dev()
        self.dev = [dev(self.ptab), i32(self.plens), i32(self.start), dev(self.table) if self.table is not None else None,
                    i32(self.lens) if self.lens is not None else None]
        return echo.make_prefix_attention_args(self.qd, self.rows, *self.dev, self.Hkv, self.scale, self.out, self.lse, self.ws,
                                               fmt=self.fmt, block_tokens=self.bs, dev_status=self.status if stat else None,
                                               k_shift=self.k_shift, v_shift=self.v_shift)

    def want(self):
        rows = []
        for b in range(self.B):
            for j in range(self.n_q):
                for hq in range(self.Hq):
                    h, k, v = hq // self.G, np.zeros((0, self.D)), np.zeros((0, self.D))
                    parts = []
                    g = self.group(b)
                    if g is not None:
                        parts.append((self.ptab, g, self.plens[g]))
                    if self.lens is not None:
                        parts.append((self.table, b, max(0, self.lens[b] - (self.n_q - 1 - j))))
                    for tab, i, n in parts:
                        kk, vv, held = mr.tokens_of(self.c, tab, i, h, n)
                        k, v = np.concatenate([k, kk[held]]), np.concatenate([v, vv[held]])
                    rows.append((k * 2.0 ** -self.k_shift, v * 2.0 ** -self.v_shift))
        r = ref.attention(self.q.reshape(-1, self.D), rows, self.scale)
        shape = (self.B, self.n_q, self.Hq)
        return [x.reshape(shape + x.shape[1:]) for x in r], np.array([len(k) for k, _ in rows]).reshape(shape)

    def check(self):
        want, n = self.want()
        # beside the additions that attention_bounds counts: a piece's sums are scaled and added up once
        # more for each of up to 160 pieces, by the merge and where the maximum moves (2^-22 each)
        far, far_lse = ref.attention_bounds(self.fmt, self.D, n + 700, *want)
        got = self.out.double().cpu().numpy()
        live = np.isfinite(want[1])
        assert int(self.status) == 0
        assert (got[~live] == 0).all()
        err = np.abs(got - want[0])
        assert (err <= far).all(), (err - far).max()
        if self.lse is not None:
            lse = self.lse.double().cpu().numpy()
            assert (lse[~live] == -np.inf).all()
            assert (np.abs(lse - want[1]) <= far_lse)[live].all()

    def run(self, **kw):
        echo.echo_prefix_attention(self.args(**kw))
        self.check()
        return self


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D,bs", [(128, 64), (64, 16), (128, 48), (64, 128), (128, 16), (64, 80)])
@pytest.mark.parametrize("plen", [1, 15, 127, 128, 129, 300])
def test_lengths_and_blocks(fmt, D, bs, plen):
    Shared(fmt, D, bs, 8, 2, 1, [plen], [0, 3], [1, 20, 140]).run()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("Hq,Hkv,n_q", [(1, 1, 1), (3, 3, 2), (10, 2, 4), (16, 1, 3), (8, 8, 1)])
def test_heads_groups_and_draft_tokens(fmt, Hq, Hkv, n_q):
    """Several groups, an empty one, a prefix of length zero, requests outside the groups."""
    lens = [n_q, 30, 5, 77, 1, 16, 0, 40, 9]
    Shared(fmt, 64, 16, Hq, Hkv, n_q, [140, 60, 0, 33], [1, 3, 3, 5, 8], lens, seed=1).run()
    Shared(fmt, 128, 32, Hq, Hkv, n_q, [260], [0, 9], lens, seed=2).run(lse=False)


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("rows", [127, 128, 129, 255, 256, 257, 400])
def test_row_tiles(fmt, rows):
    """Query rows of a KV head around the sizes of a sub-tile and a tile."""
    Shared(fmt, 64, 64, 1, 1, 1, [200], [0, rows], None, B=rows, seed=rows).run()
    Shared(fmt, 128, 64, 1, 1, 1, [130], [0, rows], [3] * rows, seed=rows + 1).run()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_no_own_tokens_tables_per_head_gaps_and_scales(fmt):
    Shared(fmt, 64, 16, 8, 2, 1, [300, 40], [0, 2, 5], None, B=6, seed=3).run()
    Shared(fmt, 64, 16, 8, 2, 2, [300, 40], [0, 2, 5], [10, 50, 3, 2, 40], heads=True, pheads=True, seed=4).run()
    Shared(fmt, 128, 16, 8, 2, 2, [500], [0, 3], [100, 50, 80], pgaps=0.4, gaps=0.3, seed=5).run()
    Shared(fmt, 64, 32, 4, 2, 1, [300], [0, 2], [10, 50], scale=-0.2, seed=6).run()
    Shared(fmt, 64, 32, 4, 2, 1, [300], [0, 2], [10, 50], scale=0.0, seed=7).run()
    Shared(fmt, 128, 32, 4, 2, 1, [700], [0, 2], [10, 50], qscale=30.0, seed=8).run()       # one key takes nearly all


def test_shifts():
    Shared(FP4, 128, 32, 8, 2, 1, [300], [0, 2], [10, 50], k_shift=3, v_shift=-2, seed=9).run()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D", [64, 128])
def test_long_prefixes_in_pieces(fmt, D):
    """Tiles cut into many pieces, and more tiles than CTAs, so that a CTA changes tiles."""
    Shared(fmt, D, 64, 4, 2, 1, [9000], [0, 3], [5, 200, 1], seed=10).run()
    Shared(fmt, D, 64, 16, 8, 1, [200, 300, 150, 129, 128, 64, 500, 257, 90, 10, 700, 33], list(range(0, 13)), [3] * 12, seed=11).run()
    g = 45
    Shared(fmt, D, 16, 4, 4, 1, [100 + 7 * i for i in range(g)], list(range(0, g + 1)), None, B=g, seed=12).run()


def test_rising_scores():
    """Keys whose scores rise from chunk to chunk by more than the slack of the running maximum: the
    output in tensor memory is rescaled again and again; and one that falls."""
    for fmt in (BF16, FP4):
        for sign in (1, -1):
            x = Shared(fmt, 64, 64, 4, 2, 1, [1200], [0, 2], [9, 30], seed=13)
            k = x.c.k.copy()
            for i in range(x.ptab.shape[1]):
                for h in range(2):
                    k[x.ptab[0, i] * 2 + h] += sign * (i - 9) * 0.5 * np.sign(x.q[0, 0, 2 * h])
            rows, kv, vv = mr.pack_rows(fmt, 64, 64, ref.bf16_round(k), x.c.v)
            x.c.rows, x.c.k, x.c.v = rows, kv, vv
            x.q *= 4
            x.run()


def test_equals_attention_over_the_joined_context():
    """The same numbers as echo_block_attention over tables that hold the prefix and the own blocks, up
    to both calls' bounds (prefixes that end with a block)."""
    for fmt in (BF16, FP4):
        x = Shared(fmt, 128, 32, 8, 2, 2, [320], [0, 4], [40, 33, 2, 64], seed=14).run()
        joined = np.concatenate([np.repeat(x.ptab, 4, 0), x.table], 1).astype(np.int32)
        out, lse = torch.empty_like(x.out), torch.empty_like(x.lse)
        echo.echo_block_attention(echo.make_block_attention_args(x.qd, x.rows, dev(joined), i32([320 + n for n in x.lens]), 2, x.scale,
                                                                 out, lse, echo.BlockAttentionWorkspace(8, 128), fmt=fmt, block_tokens=32))
        want, n = x.want()
        far, far_lse = ref.attention_bounds(fmt, 128, n + 700, *want)
        assert (np.abs((out.double() - x.out.double()).cpu().numpy()) <= 2 * far).all()
        assert (np.abs((lse.double() - x.lse.double()).cpu().numpy()) <= 2 * far_lse).all()


def test_values_that_are_not_finite():
    """A prefix value that is NaN: its dimension in the heads that share the KV head, and no other; a key
    that is NaN: whole rows of those heads."""
    for fmt, rows in ((BF16, [5, 40, 129]), (FP4, [5, 40, 129])):
        for part in (0, 1):
            x = Shared(fmt, 64, 16, 4, 2, 1, [200], [0, 2], [10, 30], seed=15)
            clean = x.run().out.clone()
            r, o = mr.row_of(x.ptab, 2, 0, 1, 150 // 16), 150 % 16
            t = ref.token_bytes(fmt, 16, 64, o)
            place = (t[part][6:8] if fmt == BF16 else t[1 + 2 * part][:1])      # dim 3; the scale of dims 0-15
            x.c.rows[r, place] = 0xFF
            echo.echo_prefix_attention(x.args())
            got, was = x.out.double().cpu().numpy(), clean.double().cpu().numpy()
            assert (got[:, :, :2] == was[:, :, :2]).all()
            if part == 0:
                assert np.isnan(got[:, :, 2:]).all()
            else:
                dims = [3] if fmt == BF16 else list(range(16))
                assert np.isnan(got[:, :, 2:, dims]).all()
                rest = [d for d in range(64) if d not in dims]
                assert (got[:, :, 2:, rest] == was[:, :, 2:, rest]).all()


def test_results_do_not_depend_on_timing():
    x = Shared(BF16, 128, 64, 16, 4, 1, [3000, 500], [0, 20, 33], [50] * 34, seed=16)
    a = x.args()
    echo.echo_prefix_attention(a)
    first = x.out.clone()
    for _ in range(20):
        x.out.fill_(0)
        echo.echo_prefix_attention(a)
        assert torch.equal(x.out, first)


def test_bad_ids_lengths_and_groups_are_flagged():
    x = Shared(BF16, 64, 16, 4, 2, 1, [64], [0, 2], [10, 30], seed=17)
    a = x.args()
    x.dev[0][0, 1] = 100000
    echo.echo_prefix_attention(a)
    assert int(x.status) == echo.DEV_BAD_INDEX
    held = np.ones(64, bool)
    held[16:32] = False
    x.ptab = x.ptab.copy()
    x.ptab[0, 1] = -1                 # answered as a block that is not held
    x.status.zero_()
    x.check()
    for i, bad in ((1, [65]), (2, [0, 3]), (2, [-1, 2])):
        x.args()
        a = echo.make_prefix_attention_args(x.qd, x.rows, *[i32(bad) if k == i else t for k, t in enumerate(x.dev)], 2, x.scale, x.out,
                                            x.lse, x.ws, block_tokens=16, dev_status=x.status)
        echo.echo_prefix_attention(a)
        assert int(x.status) == echo.DEV_BAD_INDEX, bad


def test_binding_refuses():
    x = Shared(BF16, 64, 16, 4, 2, 1, [64], [0, 2], [10, 30], seed=18)
    x.args()
    ok = dict(q=x.qd, rows=x.rows, prefix_table=x.dev[0], prefix_len=x.dev[1], group_start=x.dev[2], table=x.dev[3], ctx_len=x.dev[4],
              n_kv_heads=2, scale=0.1, out=x.out, lse=x.lse, ws=x.ws, block_tokens=16)
    echo.echo_prefix_attention(echo.make_prefix_attention_args(**ok))
    for bad in (dict(group_start=i32([0])), dict(prefix_len=i32([1, 2])), dict(prefix_table=i32([[0], [1]])), dict(block_tokens=32),
                dict(q=x.qd.float()), dict(out=x.out[:1]), dict(lse=x.lse.double()), dict(ctx_len=i32([1]))):
        with pytest.raises(echo.EchoError):
            echo.make_prefix_attention_args(**{**ok, **bad})
    for bad in (dict(table=None), dict(out=x.qd), dict(ws=echo.PrefixAttentionWorkspace(1, 1, 4, 2, 64))):
        with pytest.raises(echo.EchoError):
            echo.echo_prefix_attention(echo.make_prefix_attention_args(**{**ok, **bad}))
