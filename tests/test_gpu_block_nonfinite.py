"""echo_block_attention where queries, keys or values are not finite: what a row that sees
them answers, and that no other row notices."""
import numpy as np
import pytest
import torch

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo
from test_gpu_block_attention import BF16, FORMATS, FP4, WIDE, Attn

pytestmark = pytest.mark.gpu
# contexts and table entries: a cluster for each (request, KV head), and the line that is cut
# and merged in a second kernel
PATHS = [([40, 700], None), ([1500], None), ([900, 0, 2300], WIDE // 64)]


class Bad(Attn):
    def places(self, p, b=0, h=0):
        """Row and byte places of the key and of the value of token p: all of them in bf16, the
        scales in 4 bits (the only part that can be NaN); 0xFF there is NaN."""
        row = self.row(b, h, p // self.bs)
        t = ref.token_bytes(self.fmt, self.bs, self.D, p % self.bs)
        return row, *((t[0], t[1]) if self.fmt == BF16 else (t[1], t[3]))

    def run(self, nan):
        """One call: rows where `nan` [B][n_q][Hq] holds are NaN throughout, the others are as if
        nothing were there.  (The reference knows the values as they were first written.)"""
        echo.echo_block_attention(self.args())
        torch.cuda.synchronize()
        out, lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        assert np.isnan(out[nan]).any(-1).all()
        n, want = self.want()
        far, far_lse = ref.attention_bounds(self.fmt, self.D, n, *want)
        ok = ~nan
        assert (np.abs(out - want[0]) <= far)[ok].all()
        live = np.isfinite(want[1])
        assert (lse[ok & ~live] == -np.inf).all()
        assert (np.abs(lse - np.where(live, want[1], 0)) <= far_lse)[ok & live].all()
        return out, lse


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("lens,cap", PATHS)
def test_a_nan_query_is_not_an_empty_row(fmt, D, lens, cap):
    """lse = -inf says that a row sees no token; a row whose scores are all NaN has lse = NaN."""
    a = Bad(fmt, D, 64, 8, 2, 1, lens, seed=2, cap=cap)
    a.q[:, :, 3, 5] = float("nan")
    nan = np.zeros((a.B, 1, 8), bool)
    nan[a.lens > 0, :, 3] = True
    out, lse = a.run(nan)
    assert np.isnan(lse[nan]).all() and np.isnan(out[nan]).all()


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("lens,cap", PATHS)
@pytest.mark.parametrize("first,count", [(0, 64), (30, 1)])
def test_nan_keys_reach_the_lse(fmt, D, lens, cap, first, count):
    """A whole part of the stream with nothing but NaN scores is not a part without tokens."""
    a = Bad(fmt, D, 64, 4, 2, 1, lens, seed=3, cap=cap)
    for p in range(first, min(first + count, lens[0])):
        row, k, _ = a.places(p, 0, 1)
        a.rows_np[row, k] = 0xFF
    a.dev()
    nan = np.zeros((a.B, 1, 4), bool)
    nan[0, :, 2:] = True
    out, lse = a.run(nan)
    assert np.isnan(lse[nan]).all() and np.isnan(out[nan]).all()


# query heads, KV heads, query tokens: 8, 16, 24 and 32 rows of a KV head, and row groups beside
# the one whose queries see the token
DRAFTS = [(8, 2, 2), (6, 2, 5), (6, 1, 4), (8, 1, 4), (8, 1, 9), (2, 1, 64)]


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,n_q", DRAFTS)
@pytest.mark.parametrize("window,cap", [(0, None), (100, None), (100, WIDE // 16)])
def test_values_of_draft_tokens_stay_with_the_queries_that_see_them(fmt, D, Hq, Hkv, n_q, window, cap):
    """NaN and infinite values of the last tokens, and of the first token of the first query's
    window: the queries that do not see such a token are as if it were any other."""
    a = Bad(fmt, D, 16, Hq, Hkv, n_q, [300, 77], sinks=3 if window else 0, window=window, seed=n_q, cap=cap)
    G, bad = Hq // Hkv, np.zeros((2, n_q, Hq, D), bool)   # entries that depend on such a value
    for b, n in enumerate([300, 77]):
        first = max(0, n - (n_q - 1) - window) if window else None
        for i, p in enumerate(x for x in (n - 1, n - 2, first) if x is not None):
            row, _, v = a.places(p, b, Hkv - 1)
            what = np.zeros(D, bool)
            if fmt == BF16:
                bits = a.rows_np[row, v].view(np.uint16).copy()
                for d, x in ((3 + i, 0x7F80), (D // 2 + i, 0xFF80), (D - 1 - i, 0x7FC0)):   # inf, -inf, NaN
                    bits[d], what[d] = x, True
                a.rows_np[row, v] = bits.view(np.uint8)
            else:
                group = (i + n_q) % (D // 16)
                a.rows_np[row, v[group]] = [0x7F, 0xFF][i % 2]
                what[16 * group:16 * group + 16] = True
            for j in range(n_q):
                if a.sees(b, j, p):
                    bad[b, j, Hq - G:] |= what
    a.dev()
    echo.echo_block_attention(a.args())
    torch.cuda.synchronize()
    out, lse = a.out.double().cpu().numpy(), a.lse.double().cpu().numpy()
    n, want = a.want()
    far, far_lse = ref.attention_bounds(fmt, D, n, *want)
    live = np.isfinite(want[1])
    assert (lse[~live] == -np.inf).all() and (np.abs(lse - np.where(live, want[1], 0)) <= far_lse)[live].all()
    assert int(a.status) == 0 and (~bad).any() and bad.any()
    assert np.array_equal(np.isfinite(out), ~bad)
    assert (np.abs(np.where(bad, 0, out) - want[0]) <= far)[~bad].all()


@pytest.mark.parametrize("fmt,D", FORMATS)
def test_a_nan_key_of_a_draft_token(fmt, D):
    a = Bad(fmt, D, 16, 8, 2, 3, [300, 40], seed=9)
    row, k, _ = a.places(299, 0, 1)
    a.rows_np[row, k] = 0xFF
    a.dev()
    nan = np.zeros((2, 3, 8), bool)
    nan[0, 2, 4:] = True
    out, lse = a.run(nan)
    assert np.isnan(lse[nan]).all() and np.isnan(out[nan]).all()
