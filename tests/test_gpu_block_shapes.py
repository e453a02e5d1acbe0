"""echo_block_attention over forms of the kernel and of its merge that the other files do not
reach: many cut contexts for every count of rows, many query rows and query tokens, 4-bit rows
past 4 GiB, captures with copies and joined streams before the call."""
import numpy as np
import pytest
import torch

import sparse_attention_kv_fp8_gb300 as echo
from test_gpu_block_attention import BF16, FORMATS, FP4, WIDE, Attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("rows", [8, 16, 21, 32, 40])
def test_many_contexts_cut_into_pieces(fmt, D, rows):
    """More than half as many (request, KV head)s as CTAs: the merge finds its work by the CTA in
    which a context begins.  Short ragged contexts, empty ones, two that span several CTAs; 40
    query rows are two row groups."""
    lens = [int(x) for x in np.random.default_rng(rows).integers(0, 40, 100)]
    lens[3], lens[50], lens[51], lens[99] = 1400, 0, 777, 300
    assert 2 * len(lens) > torch.cuda.get_device_properties(0).multi_processor_count
    a = Attn(fmt, D, 16, rows, 1, 1, lens, seed=rows + D, cap=WIDE // 16)
    echo.echo_block_attention(a.args())
    a.check()


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,n_q", [(97, 1, 1), (128, 2, 2), (5, 1, 20), (2, 2, 33), (8, 1, 64), (64, 1, 16)])
@pytest.mark.parametrize("window,cap", [(0, None), (90, WIDE // 32)])
def test_many_query_rows_and_tokens(fmt, D, Hq, Hkv, n_q, window, cap):
    """33 to 1024 rows of a KV head in up to 32 row groups, up to 64 query tokens, contexts
    shorter than the query tokens among them."""
    a = Attn(fmt, D, 32, Hq, Hkv, n_q, [230, 9, 64], sinks=2 if window else 0, window=window, seed=Hq, cap=cap)
    echo.echo_block_attention(a.args())
    a.check()


def test_4_bit_rows_past_4_gib():
    a = Attn(FP4, 128, 64, 8, 2, 1, [500, 200], seed=15)
    R = echo.block_row_elems(FP4, 64, 128)
    n = 5 * (1 << 30) // (2 * R) // 2 * 2
    big = torch.empty(n, R, dtype=torch.int16, device="cuda")
    tail = a.rows.shape[0]
    assert tail % 2 == 0
    big[-tail:].copy_(a.rows)
    t = torch.where(a.t >= 0, a.t + (n - tail) // 2, -1).to(torch.int32)
    echo.echo_block_attention(a.args(rows=big, table=t))
    a.check()


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("cap", [None, WIDE // 64])
def test_captured_after_copies_and_a_joined_stream(fmt, D, cap):
    """The first call of a graph comes after a copy, a fill and the end of another stream's work,
    and its outputs are copied on: what a serving loop captures around it."""
    a = Attn(fmt, D, 64, 8, 2, 1, [900, 0, 130], seed=21, cap=cap)
    staged, zero = a.q.clone(), torch.zeros_like(a.ctx)
    lens, result = a.ctx.clone(), torch.empty_like(a.out)
    echo.echo_block_attention(a.args())
    torch.cuda.synchronize()
    main, side, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a.ctx.copy_(zero + lens)
        a.q.copy_(staged)
        a.out.fill_(float("nan"))
        main.wait_stream(side)
        echo.echo_block_attention(a.args())
        result.copy_(a.out)
        echo.echo_block_attention(a.args())
    for _ in range(3):
        a.q.zero_(), a.ctx.zero_(), a.out.zero_(), result.zero_()
        g.replay()
        a.check()
        assert torch.equal(result, a.out)
