"""echo_block_attention on bf16 rows against the bound of softmax weights that enter the value
product as two bf16 terms."""
import numpy as np
import pytest

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo
from test_gpu_block_attention import BF16, WIDE, Attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [8, 16, 24, 32])
@pytest.mark.parametrize("cap", [None, WIDE // 16])
def test_bf16_weights_enter_as_two_terms(D, rows, cap):
    """Values that nearly cancel: one bf16 term a weight would be off by several times the bound
    (test_block_bounds.py shows it)."""
    lens = [2, 6, 40, 130]
    a = Attn(BF16, D, 16, rows, 1, 1, lens, seed=rows, qscale=0.02, cap=cap)
    for b, n in enumerate(lens):
        v = ref.opposite_values(np.random.default_rng(n + D), n, D)
        for p in range(n):
            row = a.row(b, 0, p // 16)
            a.kv[row, p % 16] = ref.write_token(a.rows_np[row], BF16, 16, D, p % 16, a.kv[row, p % 16][0], v[p])
    a.dev()
    echo.echo_block_attention(a.args())
    a.check()
    n, want = a.want()
    assert (np.abs(a.out.double().cpu().numpy() - want[0]) <= ref.two_term_bounds(D, n, *want)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n_q,window", [(8, 1, 1, 0), (20, 2, 3, 0), (32, 1, 1, 100), (8, 2, 2, 64)])
@pytest.mark.parametrize("cap", [None, WIDE // 16])
def test_ordinary_bf16_calls_hold_the_two_term_bound(D, Hq, Hkv, n_q, window, cap):
    a = Attn(BF16, D, 16, Hq, Hkv, n_q, [700, 33, 0, 5], window=window, seed=Hq, cap=cap)
    echo.echo_block_attention(a.args())
    a.check()
    n, want = a.want()
    assert (np.abs(a.out.double().cpu().numpy() - want[0]) <= ref.two_term_bounds(D, n, *want)).all()
