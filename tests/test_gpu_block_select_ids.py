"""echo_block_select and table entries outside the cache's rows: not held, and flagged."""
import numpy as np
import pytest
import torch

import more_ref as mr
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev

pytestmark = pytest.mark.gpu


def check(table, lens, Hkv, n_q, k, first, last, n_rows, flagged, bs=16, seed=0):
    """Blocks whose row is outside `n_rows` (0: outside what 31 bits count) are as good as not held."""
    g = np.random.default_rng(seed)
    B, n = table.shape[0], table.shape[-1]
    x = g.standard_normal((B, n_q, Hkv, n)).astype(np.float32)
    sel, rows = (torch.full((B, n_q, Hkv, k), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    echo.echo_block_select(echo.make_block_select_args(torch.from_numpy(x).cuda(), dev(np.array(lens, np.int32)), sel, block_tokens=bs,
                                                       first=first, last=last, table=dev(table), sel_rows=rows, dev_status=st,
                                                       n_rows=n_rows))
    got, got_rows = sel.cpu().numpy(), rows.cpu().numpy()
    end = n_rows or (1 << 31) - 1
    for b in range(B):
        for j in range(n_q):
            nb = -(-max(0, lens[b] - (n_q - 1 - j)) // bs)
            for h in range(Hkv):
                at = [mr.row_of(table, Hkv, b, h, i) for i in range(nb)]
                want = mr.select(x[b, j, h].astype(np.float64), nb, k, first, last, [0 <= r < end for r in at])
                assert list(got[b, j, h]) == want, (b, j, h)
                assert list(got_rows[b, j, h]) == [at[i] if i >= 0 else -1 for i in want], (b, j, h)
    assert int(st) == (echo.DEV_BAD_INDEX if flagged else 0)


@pytest.mark.parametrize("n", [20, 300, 700, 3000])
@pytest.mark.parametrize("bad", [1 << 29, (1 << 28) + 3, (1 << 31) - 1, ((1 << 31) - 1) // 8 + 1])
def test_ids_whose_rows_wrap(n, bad):
    """Without the number of rows: ids whose row does not fit 31 bits, some of which would wrap to a row
    that exists; first, last and in between."""
    g = np.random.default_rng(n)
    table = g.integers(0, 1000, (2, n)).astype(np.int32)
    table[0, [0, 3, n // 2, n - 1]] = bad
    table[1, n // 3] = -1
    check(table, [n * 16, n * 16 - 30], 8, 2, 9, 1, 2, 0, True)


def test_the_last_id_that_has_a_row():
    """2^31 - 1 rows of 8 heads: id 2^28 - 1 has one for heads 0 to 6, and not for head 7."""
    table = np.arange(30, dtype=np.int32)[None].copy()
    table[0, 4] = (1 << 28) - 2
    check(table, [480], 8, 1, 30, 0, 0, 0, False)
    table[0, 4] = (1 << 28) - 1
    check(table, [480], 8, 1, 30, 0, 0, 0, True)


@pytest.mark.parametrize("heads", [False, True])
@pytest.mark.parametrize("n", [20, 700])
def test_ids_outside_the_rows_given(n, heads):
    g = np.random.default_rng(n)
    Hkv, n_rows = 3, 1000                          # a last block with one row of three
    shape = (2, Hkv, n) if heads else (2, n)
    top = n_rows if heads else 333
    table = g.integers(0, top, shape).astype(np.int32)
    check(table, [n * 16, 33], Hkv, 3, 12, 1, 1, n_rows, False)
    table[0, ..., n // 2] = top
    check(table, [n * 16, 33], Hkv, 3, 12, 1, 1, n_rows, True)
    check(table, [n * 16, 33], Hkv, 3, 12, 1, 1, 0, False)       # not given: the reader of the rows looks
    table[...] = 5
    table[1, ..., 3:] = 2000                       # past the length: anything
    check(table, [n * 16, 33], Hkv, 3, 12, 1, 1, n_rows, False)
    table[..., 0] = 1 << 30
    check(table, [n * 16, 33], Hkv, 3, 12, 1, 1, n_rows, True)


def test_fewer_rows_than_heads():
    table = np.zeros((1, 4), np.int32)
    check(table, [64], 5, 1, 4, 1, 0, 3, True)      # heads 3 and 4 have no row


def test_the_attention_that_reads_them_sees_no_wrapped_row():
    """An id that would wrap to row h of block 0: not selected, and the attention reads what is left."""
    g = np.random.default_rng(4)
    D, bs, Hkv, Hq = 64, 16, 8, 16
    c = mr.Cache(echo.BLOCK_BF16, bs, D, Hkv, 4, g)
    table = np.array([[1, 1 << 29, 2]], np.int32)
    q = torch.from_numpy(g.standard_normal((1, 1, Hq, D)).astype(np.float32)).bfloat16().cuda()
    scores = torch.zeros(1, 1, Hkv, 3, device="cuda")
    sel, rows = (torch.full((1, 1, Hkv, 3), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    ctx = dev(np.array([48], np.int32))
    echo.echo_block_select(echo.make_block_select_args(scores, ctx, sel, block_tokens=bs, last=1, table=dev(table), sel_rows=rows))
    out, lse = torch.zeros_like(q), torch.zeros(1, 1, Hq, device="cuda")
    for s, r in ((sel, rows), (torch.tensor([0, 2, -1], dtype=torch.int32, device="cuda").expand(1, 1, Hkv, 3).contiguous(), None)):
        if r is None:
            first, was = out.clone(), lse.clone()
            r = torch.stack([torch.tensor([8 + h, 16 + h, -1], dtype=torch.int32) for h in range(Hkv)]).cuda()[None, None]
        echo.echo_block_attention(echo.make_block_attention_args(q, c.dev(), r[:, 0].contiguous(), ctx, Hkv, 0.125, out, lse,
                                                                 echo.BlockAttentionWorkspace(2, D), block_tokens=bs,
                                                                 sel=s[:, 0].contiguous()))
    assert torch.equal(first, out) and torch.equal(was, lse)
