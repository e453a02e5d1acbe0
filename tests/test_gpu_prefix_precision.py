"""echo_prefix_attention on bf16 rows against the bound that holds the decode attention: softmax weights
that enter the value product as two bf16 terms."""
import numpy as np
import pytest

import block_ref as ref
import more_ref as mr
import sparse_attention_kv_fp8_gb300 as echo
from test_gpu_prefix_attention import BF16, Shared, pytestmark  # noqa: F401


def check(x, pieces):
    """pieces: how often a row's sums may be scaled and added up once more, by the merge and where the
    maximum moves (2^-22 each, 4 of the units that two_term_bounds counts four of for each token)."""
    echo.echo_prefix_attention(x.args())
    x.check()
    want, n = x.want()
    err = np.abs(x.out.double().cpu().numpy() - want[0])
    far = ref.two_term_bounds(x.D, n + pieces, *want)
    assert (err <= far).all(), (err - far).max()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("own", [None, [3, 17]])
@pytest.mark.parametrize("n", [2, 6, 40, 130, 300])
def test_weights_enter_as_two_terms(D, own, n):
    """Values that nearly cancel: one bf16 term a weight would be off by several times the bound."""
    x = Shared(BF16, D, 16, 8, 1, 1, [n], [0, 2], own, B=2, qscale=0.02, seed=n + D)
    v = ref.opposite_values(np.random.default_rng(n + D), n, D)
    for p in range(n):
        row = mr.row_of(x.ptab, 1, 0, 0, p // 16)
        x.c.k[row, p % 16], x.c.v[row, p % 16] = ref.write_token(x.c.rows[row], BF16, 16, D, p % 16, x.c.k[row, p % 16], v[p])
    check(x, 8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n_q,plens,start,lens,pieces", [
    (8, 1, 1, [700], [0, 3], [30, 5, 100], 12), (20, 2, 3, [140, 60, 0], [0, 2, 3, 3], [9, 200, 33, 5], 12),
    (32, 1, 1, [9000], [0, 12], [1] * 12, 700), (64, 1, 1, [300, 1000], [0, 5, 9], [40] * 10, 24)])
def test_ordinary_calls_hold_the_two_term_bound(D, Hq, Hkv, n_q, plens, start, lens, pieces):
    check(Shared(BF16, D, 16, Hq, Hkv, n_q, plens, start, lens, seed=Hq), pieces)


def test_maxima_that_move():
    """Keys whose scores rise from chunk to chunk: the output in tensor memory is rescaled again and again."""
    x = Shared(BF16, 64, 64, 4, 2, 1, [1200], [0, 2], [9, 30], seed=13)
    k = x.c.k.copy()
    for i in range(x.ptab.shape[1]):
        for h in range(2):
            k[x.ptab[0, i] * 2 + h] += (i - 9) * 0.5 * np.sign(x.q[0, 0, 2 * h])
    x.c.rows, x.c.k, x.c.v = mr.pack_rows(BF16, 64, 64, ref.bf16_round(k), x.c.v)
    x.q *= 4
    check(x, 24)
