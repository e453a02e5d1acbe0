"""The block calls that select, weigh, evict and share, run together with the others as a serving
loop uses them: block-sparse decode and prefill over selected blocks, selections that a recall makes
resident, a cache kept at a budget, captured graphs, other streams."""
import numpy as np
import pytest
import torch

import block_ref as ref
import more_ref as mr
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev, pinned_host_pool
from sparse_attention_kv_fp8_gb300 import workload as wl
from test_gpu_prefix_attention import Shared

pytestmark = pytest.mark.gpu
BF16, FP4 = echo.BLOCK_BF16, echo.BLOCK_FP4
i32 = lambda x: dev(np.array(x, np.int32))
e32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")


class Sparse:
    """One layer's block-sparse attention: argument blocks built once."""

    def __init__(self, fmt, D, bs, Hq, Hkv, n_q, lens, k, first, last, seed=0, spare=0):
        g = np.random.default_rng(seed)
        B = len(lens)
        self.__dict__.update(D=D, bs=bs, Hq=Hq, Hkv=Hkv, n_q=n_q, lens=lens, k=k, fmt=fmt, B=B)
        self.table, n = mr.tables(np.array(lens) + spare, bs, Hkv, g)
        self.c = mr.Cache(fmt, bs, D, Hkv, n, g)
        self.q = torch.from_numpy(g.standard_normal((B, n_q, Hq, D)).astype(np.float32)).bfloat16().cuda()
        self.rows, self.t, self.ctx = self.c.dev(), dev(self.table), i32(lens)
        self.summary = torch.zeros(self.rows.shape[0], 2, D, dtype=torch.bfloat16, device="cuda")
        self.scores = torch.full((B, n_q, Hkv, self.table.shape[1]), -np.inf, device="cuda")
        self.sel, self.sel_rows, self.len = e32(B, n_q, Hkv, k), e32(B, n_q, Hkv, k), e32(B, n_q)
        self.out, self.lse = torch.empty_like(self.q), torch.empty(B, n_q, Hq, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        s = D ** -0.5
        fold = lambda x: x.view(B * n_q, *x.shape[2:])
        self.calls = [
            (echo.echo_block_summary, echo.make_block_summary_args(self.rows, self.t, self.ctx, Hkv, self.summary, fmt=fmt, block_tokens=bs,
                                                                   dev_status=self.st)),
            (echo.echo_block_scores, echo.make_block_scores_args(self.q, self.summary, self.t, self.ctx, Hkv, s, self.scores, block_tokens=bs,
                                                                 dev_status=self.st)),
            (echo.echo_block_select, echo.make_block_select_args(self.scores, self.ctx, self.sel, block_tokens=bs, first=first, last=last,
                                                                 table=self.t, sel_rows=self.sel_rows, len_out=self.len, dev_status=self.st)),
            (echo.echo_block_attention, echo.make_block_attention_args(
                fold(self.q)[:, None], self.rows, fold(self.sel_rows), fold(self.len).view(-1), Hkv, s, fold(self.out)[:, None],
                fold(self.lse)[:, None], echo.BlockAttentionWorkspace(Hq // Hkv, D), fmt=fmt, block_tokens=bs, sel=fold(self.sel),
                dev_status=self.st))]

    def run(self, stream=None):
        for call, args in self.calls:
            call(args, stream=stream)

    def check(self):
        """The selection is one of the scores' best; the attention is the softmax over its tokens."""
        torch.cuda.synchronize()
        sel, scores, q = self.sel.cpu().numpy(), self.scores.double().cpu().numpy(), self.q.double().cpu().numpy()
        lens, G = self.ctx.tolist(), self.Hq // self.Hkv
        toks = []
        for b in range(self.B):
            for j in range(self.n_q):
                m = max(0, lens[b] - (self.n_q - 1 - j))
                nb = -(-m // self.bs)
                for h in range(self.Hkv):
                    a = self.calls[2][1]
                    assert list(sel[b, j, h]) == mr.select(scores[b, j, h], nb, self.k, a.first, a.last, [True] * nb)
                    k, v, _ = mr.tokens_of(self.c, self.table, b, h, m)
                    p = np.concatenate([np.arange(i * self.bs, min(m, (i + 1) * self.bs)) for i in sel[b, j, h] if i >= 0] or [np.zeros(0, int)])
                    toks += [(k[p.astype(int)], v[p.astype(int)])] * G
        want = ref.attention(q.reshape(-1, self.D), toks, self.D ** -0.5)
        far, far_lse = ref.attention_bounds(self.fmt, self.D, np.array([len(k) for k, _ in toks]), *want)
        got, lse = self.out.double().cpu().numpy().reshape(-1, self.D), self.lse.double().cpu().numpy().reshape(-1)
        live = np.isfinite(want[1])
        assert (np.abs(got - want[0]) <= far).all() and (np.abs(lse - want[1]) <= far_lse)[live].all() and int(self.st) == 0


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("n_q,lens,k", [(1, [700, 33, 1, 512], 6), (3, [400, 64, 3], 5), (40, [300], 8), (1, [100], 16)])
def test_sparse_attention(fmt, n_q, lens, k):
    """Decode, drafts and a prefill chunk, each query with blocks of its own."""
    x = Sparse(fmt, 128, 32, 8, 2, n_q, lens, k, 1, 2)
    x.run()
    x.check()


def test_all_blocks_selected_is_dense_attention():
    x = Sparse(BF16, 128, 32, 8, 2, 1, [200, 64], 7, 0, 0, seed=1)
    x.run()
    out = torch.empty_like(x.out)
    echo.echo_block_attention(echo.make_block_attention_args(x.q, x.rows, x.t, x.ctx, 2, 128 ** -0.5, out, None,
                                                             echo.BlockAttentionWorkspace(4, 128), block_tokens=32))
    assert (out.float() - x.out.float()).abs().max() <= 2.0 ** -8 * out.float().abs().max()
    x.check()


def test_captured_graph_serves_new_contents():
    """One captured step, replayed with other keys, queries and lengths."""
    x = Sparse(BF16, 64, 16, 8, 2, 2, [150, 90, 200], 5, 1, 1, seed=2, spare=60)
    x.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        x.run()
    rng = np.random.default_rng(3)
    for lens in ([150, 90, 200], [210, 3, 16], [1, 0, 255]):
        x.c = mr.Cache(BF16, 16, 64, 2, x.c.rows.shape[0] // 2, rng)
        x.rows.copy_(x.c.dev())
        x.q.copy_(torch.from_numpy(rng.standard_normal(x.q.shape).astype(np.float32)))
        x.ctx.copy_(i32(lens))
        x.scores.fill_(-np.inf)
        g.replay()
        x.check()


def test_two_streams_at_once():
    """Two layers' calls interleaved on two streams, each with workspaces of its own."""
    a, b = Sparse(BF16, 128, 32, 8, 2, 1, [3000, 700], 9, 1, 1, seed=4), Sparse(FP4, 128, 32, 8, 2, 1, [2500, 900], 9, 1, 1, seed=5)
    p = Shared(BF16, 128, 32, 8, 2, 1, [1500], [0, 3], [100, 200, 5], seed=6)
    r = Shared(FP4, 64, 32, 8, 2, 1, [900], [0, 3], [100, 200, 5], seed=7)
    pa, ra = p.args(), r.args()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(stream=s)
        echo.echo_prefix_attention(ra, stream=t)
        b.run(stream=t)
        echo.echo_prefix_attention(pa, stream=s)
    a.check(), b.check(), p.check(), r.check()


def test_prefix_attention_in_a_graph_after_its_producers():
    """The own tokens' kernel runs beside the prefix's: what comes before the call on the stream must be
    there for both.  Queries, lengths and rows are written just before, in the graph and out of it."""
    x = Shared(BF16, 128, 64, 16, 4, 1, [2000], [0, 4], [600, 300, 64, 1], seed=8)
    a = x.args()
    src = [x.qd.clone(), x.rows.clone(), x.dev[1].clone(), x.dev[4].clone()]
    dst = [x.qd, x.rows, x.dev[1], x.dev[4]]

    def step():
        for d in dst:
            d.zero_()
        for d, v in zip(dst, src):
            d.copy_(v)
        echo.echo_prefix_attention(a)

    step()
    x.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        for _ in range(3):
            step()
    for _ in range(5):
        x.out.fill_(0)
        g.replay()
    x.check()


def test_selected_blocks_recalled_from_the_host():
    """Block summaries on the device choose blocks; the rows themselves live in the host pool and a recall
    makes the chosen ones resident; attention reads them by out_slot."""
    g = np.random.default_rng(9)
    B, Hkv, Hq, D, bs, k = 2, 2, 8, 64, 16, 4
    lens = [230, 100]
    nblk = 15
    # host rows: request b, head h, block p at (b Hkv + h) nblk + p
    c = mr.Cache(BF16, bs, D, B * Hkv, nblk, g)
    order = (np.arange(nblk)[:, None] * (B * Hkv) + np.arange(B * Hkv)).T.reshape(-1)     # row ids of (head, block)
    host = pinned_host_pool(c.rows.view(np.uint16)[order])
    rows = torch.from_numpy(c.rows[order]).view(torch.int16).cuda()
    table = np.arange(B * Hkv * nblk, dtype=np.int32).reshape(B, Hkv, nblk)
    q = torch.from_numpy(g.standard_normal((B, 1, Hq, D)).astype(np.float32)).bfloat16().cuda()
    t, ctx = dev(table), i32(lens)
    summary = torch.zeros(B * Hkv * nblk, 2, D, dtype=torch.bfloat16, device="cuda")
    scores, sel = torch.full((B, 1, Hkv, nblk), -np.inf, device="cuda"), e32(B, 1, Hkv, k)
    echo.echo_block_summary(echo.make_block_summary_args(rows, t, ctx, Hkv, summary, block_tokens=bs))
    echo.echo_block_scores(echo.make_block_scores_args(q, summary, t, ctx, Hkv, 0.125, scores, block_tokens=bs))
    echo.echo_block_select(echo.make_block_select_args(scores, ctx, sel, block_tokens=bs, last=1))
    pool = echo.Pool(40, host)
    echo.echo_pool_init(pool)
    ws, slots = echo.Workspace(40, B * Hkv * k), e32(B * Hkv, 1, k)
    echo.echo_prefetch_recall(pool, ws, sel.view(B * Hkv, 1, k), t.view(B * Hkv, nblk), i32(np.repeat(-(-np.array(lens) // bs), Hkv)), 1, slots)
    out, lse = torch.empty_like(q), torch.empty(B, 1, Hq, device="cuda")
    echo.echo_block_attention(echo.make_block_attention_args(q, pool.gpu_kv, slots.view(B, Hkv, k), ctx, Hkv, 0.125, out, lse,
                                                             echo.BlockAttentionWorkspace(4, D), block_tokens=bs, sel=sel.view(B, Hkv, k)))
    got, picked = out.double().cpu().numpy(), sel.cpu().numpy()
    toks = []
    for b in range(B):
        for hq in range(Hq):
            h = hq // 4
            ids = [i for i in picked[b, 0, h] if i >= 0]
            assert len(ids) == k and -(-lens[b] // bs) - 1 in ids
            p = [(i, o) for i in ids for o in range(min(bs, lens[b] - i * bs))]
            r = order[(b * Hkv + h) * nblk + np.array([i for i, _ in p])]
            o = np.array([o for _, o in p])
            toks.append((c.k[r, o], c.v[r, o]))
    want = ref.attention(q.double().cpu().numpy().reshape(-1, D), toks, 0.125)
    far, _ = ref.attention_bounds(BF16, D, np.array([len(x) for x, _ in toks]), *want)
    assert (np.abs(got.reshape(-1, D) - want[0]) <= far).all()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_cache_kept_at_a_budget(fmt):
    """A loop of appends, attention, gathered weights and evictions, with the blocks going back to their
    stack: the tokens that stay are those of a host that follows the same weights, and attention over
    what is left is the softmax over them."""
    g = np.random.default_rng(10)
    B, Hq, Hkv, D, bs, keep, recent, sinks, maxb = 3, 4, 2, 64, 16, 40, 8, 2, 6
    T, n_blocks = maxb * bs, B * maxb
    table, free = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda"), torch.arange(n_blocks, dtype=torch.int32, device="cuda")
    count = [i32([n_blocks]), e32(1)]
    rows = torch.zeros(n_blocks * Hkv, echo.block_row_elems(fmt, bs, D), dtype=torch.int16, device="cuda")
    st, cs = torch.zeros(1, dtype=torch.int32, device="cuda"), echo.rope_table(512, 64)
    acc = [torch.zeros(B, Hkv, T, device="cuda") for _ in range(2)]
    pos = [torch.zeros(B, Hkv, T, dtype=torch.int32, device="cuda") for _ in range(2)]
    ln, nxt = np.zeros(B, np.int32), np.zeros(B, np.int32)
    kv = [[{} for _ in range(Hkv)] for _ in range(B)]             # position -> (k, v)
    slots = [[[] for _ in range(Hkv)] for _ in range(B)]          # position of each slot
    ws, ews = echo.BlockAttentionWorkspace(Hq // Hkv, D), echo.BlockEvictWorkspace(B, Hkv, keep)
    for step in range(12):
        new = np.array([30, 50, 7], np.int32) if step == 0 else np.array([1, 1, 9 if step % 3 == 0 else 1], np.int32)
        n = int(new.sum())
        slot, cpos = e32(n), e32(n)
        echo.echo_block_tables(echo.make_block_tables_args(i32(ln), i32(ln + new), bs, table, free, count[0], count[1], slot, cpos, dev_status=st))
        count.reverse()
        x = torch.from_numpy(g.standard_normal((n, Hq + 2 * Hkv, D)).astype(np.float32)).bfloat16().cuda()
        true_pos = np.concatenate([nxt[b] + np.arange(new[b]) for b in range(B)])
        o = [torch.empty(n, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
        echo.echo_qk_norm_rope(echo.make_qk_norm_rope_args(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], i32(true_pos), cs, o[0], slot_map=slot,
                                                           rows=rows, fmt=fmt, block_tokens=bs, k_out=o[1], v_out=o[2], dev_status=st))
        at = 0
        kc, vc = o[1].double().cpu().numpy(), o[2].double().cpu().numpy()
        for b in range(B):
            for i in range(new[b]):
                for h in range(Hkv):
                    kv[b][h][int(nxt[b]) + i] = (kc[at, h], vc[at, h])
                    slots[b][h].append(int(nxt[b]) + i)
                at += 1
        old = ln.copy()
        ln, nxt = ln + new, nxt + new
        q = torch.stack([o[0][int(new[:b + 1].sum()) - 1] for b in range(B)])[:, None].contiguous()
        out, lse = torch.empty_like(q), torch.empty(B, 1, Hq, device="cuda")
        ctx = i32(ln)
        echo.echo_block_attention(echo.make_block_attention_args(q, rows, table, ctx, Hkv, D ** -0.5, out, lse, ws, fmt=fmt, block_tokens=bs,
                                                                 dev_status=st))
        toks = [tuple(np.stack([kv[b][hq // 2][p][i] for p in slots[b][hq // 2]]) for i in (0, 1)) for b in range(B) for hq in range(Hq)]
        want = ref.attention(q.double().cpu().numpy().reshape(-1, D), toks, D ** -0.5)
        far, _ = ref.attention_bounds(fmt, D, np.array([len(k) for k, _ in toks]), *want)
        assert (np.abs(out.double().cpu().numpy().reshape(-1, D) - want[0]) <= far).all(), step
        echo.echo_block_weights(echo.make_block_weights_args(q, rows, table, ctx, Hkv, D ** -0.5, lse, acc[0], acc[1], old_len=i32(old),
                                                             decay=0.9, fmt=fmt, block_tokens=bs, dev_status=st))
        lo = e32(B)
        echo.echo_block_evict(echo.make_block_evict_args(rows, table, ctx, lo, Hkv, keep, acc[1], acc[0], ews, sinks=sinks, recent=recent,
                                                         pos=pos[0], pos_out=pos[1], pos_len=i32(old), next_pos=i32(nxt), fmt=fmt,
                                                         block_tokens=bs, dev_status=st))
        w = acc[1].double().cpu().numpy()
        for b in range(B):
            for h in range(Hkv):
                p = np.array(slots[b][h])
                src = mr.evict(w[b, h], p, int(ln[b]), keep, sinks, recent, int(nxt[b]))
                slots[b][h] = [int(p[i]) for i in src]
                assert pos[1][b, h, :len(src)].tolist() == slots[b][h]
        after = lo.cpu().numpy()
        assert (after == np.minimum(ln, keep)).all() and int(st) == 0
        e = e32(1)
        echo.echo_block_tables(echo.make_block_tables_args(ctx, lo, bs, table, free, count[0], count[1], e, dev_status=st))
        count.reverse()
        pos.reverse()
        ln = after.copy()
        assert int(count[0]) == n_blocks - int((-(-ln // bs)).sum())


def test_calls_on_another_stream_than_the_tensors():
    """Everything on a side stream, the tensors made on the default one."""
    x = Sparse(FP4, 64, 32, 8, 2, 1, [500, 90], 4, 1, 1, seed=11)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        x.run()
        torch.cuda.current_stream().synchronize()
    x.check()
