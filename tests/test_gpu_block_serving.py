"""The block calls run together, as a serving loop uses them: tables from lengths, norm +
rotation into the cache, attention over it -- prefill, decode, drafts taken back, finished
requests whose blocks serve new ones -- and attention over the rows a block recall made
resident.  Every step against 64-bit references."""
import numpy as np
import pytest
import torch

import block_ref as ref
import oracle
import sparse_attention_kv_fp8_gb300 as echo
from sparse_attention_kv_fp8_gb300 import workload as wl
from helpers import dev, pinned_host_pool

pytestmark = pytest.mark.gpu
BF16, FP4 = echo.BLOCK_BF16, echo.BLOCK_FP4
Hq, Hk, D, BS, RD = 8, 2, 128, 16, 64


class Loop:
    """B request slots over one cache of n_blocks blocks; the tokens' keys and values, as the
    cache holds them, are kept on the host."""

    def __init__(self, fmt, B, n_blocks, max_blocks, seed):
        self.fmt, self.B, self.g = fmt, B, torch.Generator(device="cuda").manual_seed(seed)
        i32 = lambda *n: torch.full(n, -1, dtype=torch.int32, device="cuda")
        self.table, self.free = i32(B, max_blocks), torch.arange(n_blocks, dtype=torch.int32, device="cuda")
        self.count = [torch.tensor([n_blocks], dtype=torch.int32, device="cuda"), i32(1)]
        self.rows = torch.full((n_blocks * Hk, echo.block_row_elems(fmt, BS, D)), -1, dtype=torch.int16, device="cuda")
        self.len = np.zeros(B, np.int32)
        self.cs = echo.rope_table(2048, RD)
        self.wq, self.wk = (1 + 0.1 * torch.randn(D, generator=self.g, device="cuda") for _ in range(2))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = [[] for _ in range(B)]           # per request: (k [Hk][D], v [Hk][D]) per token

    def advance(self, new, pad=4):
        """One step to the lengths `new`: returns the rotated queries of the new tokens."""
        old, new = self.len, np.array(new, np.int32)
        T = int(np.maximum(new - old, 0).sum()) + pad
        i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")
        slot, pos = i32(T), i32(T)
        echo.echo_block_tables(echo.make_block_tables_args(dev(old), dev(new), BS, self.table, self.free, self.count[0],
                                                           self.count[1], slot, pos, dev_status=self.status))
        self.count.reverse()
        x = torch.randn(T, (Hq + 2 * Hk) * D, generator=self.g, device="cuda").bfloat16()
        cut = lambda a, n: x[:, a * D:(a + n) * D].unflatten(1, (n, D))
        e = lambda h: torch.empty(T, h, D, dtype=torch.bfloat16, device="cuda")
        q, k, v = e(Hq), e(Hk), e(Hk)
        echo.echo_qk_norm_rope(echo.make_qk_norm_rope_args(
            cut(0, Hq), cut(Hq, Hk), cut(Hq + Hk, Hk), pos, self.cs, q, q_weight=self.wq, k_weight=self.wk,
            slot_map=slot, rows=self.rows, fmt=self.fmt, block_tokens=BS, k_out=k, v_out=v, dev_status=self.status))
        kc, vc, i = k.double().cpu().numpy(), v.double().cpu().numpy(), 0
        for b in range(self.B):
            del self.kv[b][max(0, int(new[b])):]
            for _ in range(int(old[b]), int(new[b])):
                self.kv[b].append((kc[i], vc[i]))
                i += 1
        # the keys themselves, against the formula (bf16 rows hold them as they are)
        want, mag = ref.norm_rope(cut(Hq, Hk).double().cpu().numpy()[:i], self.wk.double().cpu().numpy(), 1e-6,
                                  self.cs.double().cpu().numpy()[pos[:i].cpu().numpy()], RD, False)
        if self.fmt == BF16:
            assert (np.abs(kc[:i] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * mag).all()
        self.len = new
        return q

    def attend(self, q, sinks=0, window=0):
        """q [B][n_q][Hq][D] of the newest tokens, checked against the host's tokens."""
        B, n_q = q.shape[:2]
        out, lse = torch.empty_like(q), torch.empty(B, n_q, Hq, device="cuda")
        ws = echo.BlockAttentionWorkspace(n_q * (Hq // Hk), D)
        echo.echo_block_attention(echo.make_block_attention_args(q, self.rows, self.table, dev(self.len), Hk, D ** -0.5, out,
                                                                 lse, ws, fmt=self.fmt, block_tokens=BS, sinks=sinks,
                                                                 window=window, dev_status=self.status))
        got, got_lse, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
        assert int(self.status) == 0
        G = Hq // Hk
        for b in range(B):
            for j in range(n_q):
                n = int(self.len[b]) - (n_q - 1 - j)
                p = np.arange(max(n, 0))
                p = p[(p >= n - window) | (p < sinks)] if window else p
                for h in range(Hk):
                    k = np.array([self.kv[b][i][0][h] for i in p]).reshape(-1, D)
                    v = np.array([self.kv[b][i][1][h] for i in p]).reshape(-1, D)
                    hs = slice(h * G, (h + 1) * G)
                    r = ref.attention(qn[b, j, hs], [(k, v)] * G, D ** -0.5)
                    far, far_lse = ref.attention_bounds(self.fmt, D, np.full(G, len(p)), *r)
                    assert (np.abs(got[b, j, hs] - r[0]) <= far).all()
                    if len(p):
                        assert (np.abs(got_lse[b, j, hs] - r[1]) <= far_lse).all()
                    else:
                        assert (got_lse[b, j, hs] == -np.inf).all()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_a_serving_loop(fmt):
    L = Loop(fmt, B=4, n_blocks=40, max_blocks=20, seed=1)
    L.advance([37, 0, 120, 16])                                 # prefill three requests
    for _ in range(3):                                          # decode; request 1 arrives meanwhile
        new = L.len + np.array([1, 0, 1, 1], np.int32)
        q = L.advance(new, pad=0)
        full = torch.zeros(4, 1, Hq, D, dtype=torch.bfloat16, device="cuda")
        full[[0, 2, 3], 0] = q
        L.attend(full)
    L.advance([L.len[0], 90, 0, L.len[3]])                      # request 2 ends, 1 takes over its blocks
    q = L.advance(L.len + np.array([3, 3, 3, 3], np.int32), pad=0).view(4, 3, Hq, D)   # two drafts each
    L.attend(q)
    L.attend(q, sinks=2, window=20)
    L.advance(L.len - np.array([2, 0, 1, 2], np.int32))         # drafts taken back
    q = L.advance(L.len + 1, pad=0).view(4, 1, Hq, D)
    L.attend(q)
    L.attend(q, sinks=16, window=1)
    used = int((-(-L.len // BS)).sum())
    assert int(L.count[0]) == 40 - used                         # every other block is free again
    held = [int(x) for b in range(4) for x in L.table[b, :-(-int(L.len[b]) // BS)]]
    assert sorted(held + L.free[:40 - used].tolist()) == list(range(40))


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_attention_over_the_rows_a_block_recall_made_resident(fmt):
    """Two requests x 2 KV heads, blocks in the pinned host pool, 12 of each selected and
    recalled into a pool of 60 slots: the attention reads them by the recall's out_slot."""
    B, n_blocks, k, n_g = 2, 30, 12, 60
    R = echo.block_row_elems(fmt, BS, D)
    g = np.random.default_rng(2)
    rows_np, kv = np.zeros((B * Hk * n_blocks, 2 * R), np.uint8), {}
    for r in range(rows_np.shape[0]):
        for off in range(BS):
            kv[r, off] = ref.write_token(rows_np[r], fmt, BS, D, off, ref.bf16_round(g.standard_normal(D)),
                                         ref.bf16_round(g.standard_normal(D)))
    pool = echo.Pool(n_g, pinned_host_pool(rows_np.view(np.uint16)))
    echo.echo_pool_init(pool)
    ws = echo.Workspace(n_g, B * Hk * k)
    r2h = wl.req_to_host(B * Hk, n_blocks)
    ctx_blocks = np.full(B * Hk, n_blocks, np.int32)
    lens = np.array([n_blocks * BS, n_blocks * BS - 7], np.int32)
    aws = echo.BlockAttentionWorkspace(Hq // Hk, D)
    for t, sc in enumerate(wl.block_scores(B * Hk, n_blocks, 3, 3, 0.7)):
        sel = torch.empty(B * Hk, 1, k, dtype=torch.int32, device="cuda")
        kth, slots = torch.empty(B * Hk, 1, device="cuda"), torch.empty_like(sel)
        echo.echo_select_topk(dev(sc), dev(ctx_blocks), k, sel, kth)
        echo.echo_prefetch_recall(pool, ws, sel, dev(r2h), dev(ctx_blocks), t + 1, slots)
        q = torch.randn(B, 1, Hq, D, device="cuda").bfloat16()
        out, lse = torch.empty_like(q), torch.empty(B, 1, Hq, device="cuda")
        echo.echo_block_attention(echo.make_block_attention_args(
            q, pool.gpu_kv, slots.view(B, Hk, k), dev(lens), Hk, D ** -0.5, out, lse, aws, fmt=fmt, block_tokens=BS,
            sel=sel.view(B, Hk, k)))
        got, got_lse, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
        want_sel, _ = oracle.select_topk(sc, ctx_blocks, k)
        G = Hq // Hk
        for b in range(B):
            for h in range(Hk):
                tok = [kv[int(r2h[b * Hk + h, lb]), o] for lb in want_sel[b * Hk + h, 0] for o in range(BS)
                       if lb * BS + o < lens[b]]
                kk, vv = np.array([x[0] for x in tok]), np.array([x[1] for x in tok])
                r = ref.attention(qn[b, 0, h * G:(h + 1) * G], [(kk, vv)] * G, D ** -0.5)
                far, far_lse = ref.attention_bounds(fmt, D, np.full(G, len(tok)), *r)
                assert (np.abs(got[b, 0, h * G:(h + 1) * G] - r[0]) <= far).all()
                assert (np.abs(got_lse[b, 0, h * G:(h + 1) * G] - r[1]) <= far_lse).all()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_a_captured_decode_step(fmt):
    """Tables, norm + rotation and attention of a decode step captured once into a graph and
    replayed over static buffers: lengths, projections and the stack's height change between
    replays, one request pauses, one ends and starts again."""
    B, n_blocks, mb = 3, 24, 10
    g = torch.Generator(device="cuda").manual_seed(5)
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    old, new, table, count, count_out, slot, pos = z(B), z(B), z(B, mb) - 1, z(1) + n_blocks, z(1), z(B), z(B)
    free = torch.arange(n_blocks, dtype=torch.int32, device="cuda")
    status, cs = z(1), echo.rope_table(512, RD)
    x = torch.zeros(B, (Hq + 2 * Hk) * D, dtype=torch.bfloat16, device="cuda")
    cut = lambda a, n: x[:, a * D:(a + n) * D].unflatten(1, (n, D))
    e = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    q, k, v, out, lse = e(B, Hq, D), e(B, Hk, D), e(B, Hk, D), e(B, 1, Hq, D), torch.zeros(B, 1, Hq, device="cuda")
    rows = torch.full((n_blocks * Hk, echo.block_row_elems(fmt, BS, D)), -1, dtype=torch.int16, device="cuda")
    # the list of new tokens is not the list of requests (a paused one has none): the graph
    # attends with each request's newest query, gathered by cu_new
    cu, qa = z(B + 1), e(B, 1, Hq, D)
    tables = echo.make_block_tables_args(old, new, BS, table, free, count, count_out, slot, pos, cu, dev_status=status)
    rope = echo.make_qk_norm_rope_args(cut(0, Hq), cut(Hq, Hk), cut(Hq + Hk, Hk), pos, cs, q, slot_map=slot, rows=rows,
                                       fmt=fmt, block_tokens=BS, k_out=k, v_out=v, dev_status=status)
    attn = echo.make_block_attention_args(qa, rows, table, new, Hk, D ** -0.5, out, lse,
                                          echo.BlockAttentionWorkspace(Hq // Hk, D), fmt=fmt, block_tokens=BS,
                                          dev_status=status)

    def step():
        echo.echo_block_tables(tables)
        echo.echo_qk_norm_rope(rope)
        qa.copy_(q.index_select(0, cu[:B].clamp(max=B - 1).long()).unsqueeze(1))
        echo.echo_block_attention(attn)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kv, lens = [[] for _ in range(B)], np.zeros(B, np.int32)
    for t in range(40):
        nxt = lens + 1
        if t % 5 == 3:
            nxt[1] = lens[1]                    # paused
        if t == 20:
            nxt[2] = 0                          # ended: its blocks return
        old.copy_(dev(lens)), new.copy_(dev(nxt))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        count.copy_(count_out)
        kc, vc, qn = (a.double().cpu().numpy() for a in (k, v, qa))
        i = 0
        for b in range(B):
            if nxt[b] == 0:
                kv[b] = []
            elif nxt[b] > lens[b]:
                kv[b].append((kc[i], vc[i]))
                i += 1
        lens = nxt
        used = int((-(-lens // BS)).sum())
        assert int(count) == n_blocks - used and int(status) == 0
        got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(B):
            for h in range(Hk):
                hs = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
                kk = np.array([c[0][h] for c in kv[b]]).reshape(-1, D)
                vv = np.array([c[1][h] for c in kv[b]]).reshape(-1, D)
                r = ref.attention(qn[b, 0, hs], [(kk, vv)] * (Hq // Hk), D ** -0.5)
                far, far_lse = ref.attention_bounds(fmt, D, np.full(Hq // Hk, len(kk)), *r)
                assert (np.abs(got[b, 0, hs] - r[0]) <= far).all(), (t, b)
                if len(kk):
                    assert (np.abs(got_lse[b, 0, hs] - r[1]) <= far_lse).all()
                else:
                    assert (got_lse[b, 0, hs] == -np.inf).all()
