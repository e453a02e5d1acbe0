"""Contexts of nearly 2^31 tokens, and blocks of any number of them: block counts that the 31 bits of a
length do not hold on the way (echo_block_scores, echo_block_select, echo_block_summary)."""
import numpy as np
import pytest
import torch

import more_ref as mr
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [(1 << 30) - 512, (1 << 30) + 1, (1 << 31) - 1024])
@pytest.mark.parametrize("n", [1, 5000, (1 << 31) - 1024])
def test_one_block_holds_the_context(bs, n):
    g = np.random.default_rng(0)
    blocks = ((1 << 31) - 1024) // bs
    want = -(-n // bs)
    if want > blocks:
        pytest.skip("longer than the table holds")
    q = torch.from_numpy(g.standard_normal((1, 1, 2, 64)).astype(np.float32)).bfloat16().cuda()
    k = torch.from_numpy(g.standard_normal((blocks, 1, 64)).astype(np.float32)).bfloat16().cuda()
    scores = torch.full((1, 1, 1, blocks), 1234.0, device="cuda")
    table, ctx = dev(np.arange(blocks, dtype=np.int32)[None]), dev(np.array([n], np.int32))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    echo.echo_block_scores(echo.make_block_scores_args(q, torch.cat([k, k], 1), table, ctx, 1, 1.0, scores, block_tokens=bs, dev_status=st))
    # (minimum and maximum are the same key: the score of it)
    x = q[0, 0].double().cpu() @ k[:, 0].double().cpu().T
    mag = q[0, 0].double().abs().cpu() @ k[:, 0].double().abs().cpu().T
    got = scores[0, 0, 0].double().cpu()
    assert (torch.abs(got - x.amax(0)) <= 130 * 2.0 ** -23 * mag.amax(0))[:want].all() and (got[want:] == 1234.0).all() and int(st) == 0
    sel, ln = torch.full((1, 1, 1, 3), -7, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    echo.echo_block_select(echo.make_block_select_args(scores, ctx, sel, block_tokens=bs, table=table, len_out=ln, dev_status=st))
    assert sel.flatten().tolist() == (list(range(want)) + [-1] * 3)[:3] and int(ln) == n and int(st) == 0


@pytest.mark.parametrize("bs,blocks", [(1792, 1198372), (1296, 1657008), (512, (1 << 22) - 2)])
def test_summaries_of_the_longest_contexts(bs, blocks):
    """2^31 - 1024 tokens or a little less, of which three blocks are held, beside a short context."""
    g = np.random.default_rng(0)
    c = mr.Cache(echo.BLOCK_FP4, bs, 64, 1, 5, g)
    table = np.full((2, blocks), -1, np.int32)
    table[0, [0, blocks // 2, blocks - 1]] = [1, 3, 0]
    table[1, 0] = 4
    n = [blocks * bs - 7, 30]
    out, st = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    c.spoil(0, range(bs - 7, bs))
    c.spoil(4, range(30, bs))
    echo.echo_block_summary(echo.make_block_summary_args(c.dev(), dev(table), dev(np.array(n, np.int32)), 1, out, fmt=echo.BLOCK_FP4,
                                                         block_tokens=bs, dev_status=st))
    want = np.zeros((5, 2, 64))
    for r, m in ((1, bs), (3, bs), (0, bs - 7), (4, 30)):
        want[r, 0], want[r, 1] = c.k[r, :m].min(0), c.k[r, :m].max(0)
    assert (out.double().cpu().numpy() == want).all() and int(st) == 0
