"""echo_prefix_attention over 4-bit prefixes for queries of zeros, or nearly: the power of two that a row
is scaled by, times a small softmax scale, is below what fp32 holds.  Tokens that are not seen still weigh
nothing."""
import numpy as np
import pytest

import sparse_attention_kv_fp8_gb300 as echo
from test_gpu_prefix_attention import BF16, FP4, Shared, pytestmark  # noqa: F401


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("scale,k_shift", [(None, 0), (0.0, 0), (-0.0, 0), (1e-30, 0), (None, 24), (None, 32), (-0.1, 32)])
@pytest.mark.parametrize("plen,pgaps", [(300, 0.0), (1, 0.0), (500, 0.4)])
def test_queries_of_zeros(fmt, scale, k_shift, plen, pgaps):
    if fmt == BF16 and k_shift:
        pytest.skip("k_shift is for 4-bit rows")
    x = Shared(fmt, 64, 16, 8, 2, 1, [plen], [0, 2], [10, 50, 7], scale=scale, k_shift=k_shift, pgaps=pgaps, seed=21)
    x.q[0, 0, 0] = 0.0
    x.q[0, 0, 5] = 0.0
    x.q[1, 0, 1] = 2.0 ** -126 * np.sign(x.q[1, 0, 1])      # the least normal number
    x.q[1, 0, 2] = 2.0 ** -133 * np.sign(x.q[1, 0, 2])      # the least of all
    x.run()


@pytest.mark.parametrize("D", [64, 128])
def test_all_queries_zeros_no_own_tokens(D):
    x = Shared(FP4, D, 32, 4, 2, 2, [129], [0, 3], None, B=3, scale=0.0, seed=22)
    x.q[:] = 0.0
    x.run()
    lse = x.lse.cpu().numpy()
    assert np.abs(lse - np.log(129)).max() <= 1e-5
