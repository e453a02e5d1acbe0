"""echo_prefix_attention and group starts that are not ascending: flagged, and nothing is read or written
outside, also where the groups overlap so much that their tiles would not be counted in 31 bits."""
import numpy as np
import pytest
import torch

import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev
from test_gpu_prefix_attention import BF16, FP4, Shared, pytestmark  # noqa: F401

i32 = lambda x: dev(np.array(x, np.int32))


def with_groups(x, plens, start, ptab):
    """The call of `x` with other prefixes, its own tokens as they are."""
    x.args()
    return echo.make_prefix_attention_args(x.qd, x.rows, ptab, i32(plens), i32(start), *x.dev[3:], x.Hkv, x.scale, x.out, x.lse, x.ws,
                                           fmt=x.fmt, block_tokens=x.bs, dev_status=x.status)


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("groups", [2, 5, 40, 300])
def test_overlapping_groups(fmt, groups):
    """Every other group is all requests: flagged, and the next call is served as ever."""
    x = Shared(fmt, 64, 16, 8, 2, 1, [100], [0, 6], [10, 3, 50, 7, 1, 20], seed=31)
    x.args()
    ptab = x.dev[0].expand(groups, -1).contiguous()
    start = [0 if g % 2 == 0 else 6 for g in range(groups + 1)]
    a = with_groups(x, [100 - g % 9 for g in range(groups)], start, ptab)
    echo.echo_prefix_attention(a)
    assert int(x.status) == echo.DEV_BAD_INDEX
    x.run(ws=x.ws)


@pytest.mark.parametrize("own", [True, False])
def test_more_tiles_than_31_bits_count(own):
    """300 groups that are all 1200 requests by turns, 300 tiles of 47723 chunks each: 2.1e9 units, of which the
    check on disjoint groups expects 2.9e7.  Taken for no prefixes: the own tokens alone."""
    lens = [2 if b % 100 == 0 else 0 for b in range(1200)] if own else None
    x = Shared(BF16, 64, 512, 64, 1, 1, [5], [0, 0], lens, B=1200, seed=32)
    x.args()
    groups, blocks = 300, 11931
    assert groups // 2 * (1200 * 64 // 256) * (blocks * 4) >= 1 << 31
    ptab = torch.full((groups, blocks), -1, dtype=torch.int32, device="cuda")
    a = with_groups(x, [blocks * 512] * groups, [0 if g % 2 == 0 else 1200 for g in range(groups + 1)], ptab)
    echo.echo_prefix_attention(a)
    assert int(x.status) == echo.DEV_BAD_INDEX
    x.status.zero_()
    x.check()                                       # (group [0, 0): no prefix either)
