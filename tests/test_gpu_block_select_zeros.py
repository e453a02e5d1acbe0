"""echo_block_select on rows whose k-th best lies among zeros or beside them: many scores in one part of
the counted range, of both signs, so that the search for the k-th best goes on by halving."""
import numpy as np
import pytest
import torch

import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev

pytestmark = pytest.mark.gpu
TINY = float(np.float32(1e-45))


def row(g, far, counts, n):
    """n scores: one at `far` (the others then share a part of the range), counts[v] times each value v,
    the rest of them -3; shuffled."""
    x = np.concatenate([[far]] + [np.full(c, v) for v, c in counts.items()])
    x = np.concatenate([x, np.full(n - len(x), -3.0)]).astype(np.float32)
    return g.permutation(x)


def check(x, k):
    """x [rows][n]: a KV head each.  The k largest, ties to the lower block, ascending, then -1."""
    rows, n = x.shape
    sel = torch.full((1, 1, rows, k), -7, dtype=torch.int32, device="cuda")
    echo.echo_block_select(echo.make_block_select_args(torch.from_numpy(x).cuda()[None, None], dev(np.array([n * 16], np.int32)), sel,
                                                       block_tokens=16))
    want = np.full((rows, k), -1, np.int32)
    want[:, :min(n, k)] = np.sort(np.argsort(-x.astype(np.float64), axis=1, kind="stable")[:, :k], axis=1)
    got = sel[0, 0].cpu().numpy()
    wrong = np.nonzero((got != want).any(1))[0]
    assert len(wrong) == 0, (k, len(wrong), got[wrong[0]], want[wrong[0]])


@pytest.mark.parametrize("rows", [2, 700])
def test_one_warp_a_row(rows):
    """64 blocks, k = 21: the far one, ten of 1 and ten of 0."""
    g = np.random.default_rng(0)
    check(np.stack([row(g, 1000.0, {1.0: 10, 0.0: 10, -0.5: 20, -1.0: 23}, 64) for _ in range(rows)]), 21)


@pytest.mark.parametrize("far", [-3.4028234663852886e38, 1e4, 3e38])
@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_k_best_end_with_the_zeros(far, zero):
    """281 blocks, k = 160: 120 above zero and the 40 zeros (or the far one)."""
    g = np.random.default_rng(1)
    x = np.stack([row(g, far, {-2.0: 60, -1.0: 60, zero: 40, 1.0: 60, 2.0: 60}, 281) for _ in range(4)])
    for k in (120, 121, 159, 160, 161, 162, 220):
        check(x, k)


@pytest.mark.parametrize("rows", [2, 700])
@pytest.mark.parametrize("n", [40, 256, 400, 512, 900, 1024, 1500, 2048, 3001, 4096, 8192, 12345, 30000])
def test_every_width(rows, n):
    """All numbers of warps and of blocks a thread; k-th bests above, among and below the zeros, the least
    steps beside zero among the scores."""
    g = np.random.default_rng(n)
    c = n // 5
    sides = {2.0: c // 2, TINY: c // 2, 0.0: c, -TINY: c // 2, -1.0: c // 2, -2.0: c // 2, 1.0: c // 2}
    x = np.stack([row(g, 1e4 if r % 2 else -1e30, sides, n) for r in range(rows)])
    above = 3 * (c // 2)
    for k in sorted({above, above + 1, above + c - 1, above + c, above + c + 1, above + c + c // 2 + 1}):
        check(x, k)


def test_symmetric_random_rows():
    """Values of a symmetric grid in random numbers and an outlier."""
    g = np.random.default_rng(2)
    for n in (200, 300, 500):
        x = g.choice(np.array([-2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2], np.float32), (3, n))
        x[:, g.integers(0, n)] = 5e5
        for k in range(1, n + 2, 3):
            check(x, k)
