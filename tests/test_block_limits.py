"""Sizes past which a block call's counters would not fit 31 bits: refused.  No GPU needed."""
import ctypes

import pytest

import sparse_attention_kv_fp8_gb300 as echo
from test_block_abi import attn_args, lib  # noqa: F401


@pytest.mark.parametrize("bad,why", [
    # one request of 2^31 - 1024 tokens is fine by itself, 32768 KV heads of it are not
    (dict(B=16, n_heads=32768, n_kv_heads=32768, block_tokens=16, max_blocks=1 << 26), b"contexts too large"),
    (dict(B=1 << 14, n_heads=8, n_kv_heads=8, block_tokens=256, max_blocks=1 << 16), b"contexts too large"),
    # 1024 query rows are 32 row groups, each on the line
    (dict(B=1 << 10, n_q=16, n_heads=64, n_kv_heads=1, block_tokens=16, max_blocks=1 << 22), b"contexts too large"),
    (dict(n_heads=65537, n_kv_heads=65537), b"too many heads"),
])
def test_attention_refuses_what_its_counters_cannot_hold(lib, bad, why):  # noqa: F811
    assert lib.echo_block_attention(ctypes.byref(attn_args(**bad)), None) == echo.ECHO_EINVAL
    assert why in lib.echo_last_error_string(), lib.echo_last_error_string()


def test_attention_accepts_large_tables(lib):  # noqa: F811
    """Half of the limit passes this check (and is refused for its workspace, which comes later)."""
    a = attn_args(B=1 << 13, n_heads=8, n_kv_heads=8, block_tokens=256, max_blocks=(1 << 16) - 1, workspace_bytes=1)
    assert lib.echo_block_attention(ctypes.byref(a), None) == echo.ECHO_EINVAL
    assert b"smaller" in lib.echo_last_error_string(), lib.echo_last_error_string()


@pytest.mark.parametrize("rows,D,kept", [(8, 128, 8), (20, 64, 32), (1024, 128, 32)])
def test_a_workspace_holds_what_the_largest_grid_writes(lib, rows, D, kept):  # noqa: F811
    """Two CTAs on each of 152 SMs leave two partial results and a work item each, no more."""
    n = ctypes.c_size_t()
    assert lib.echo_block_attention_workspace_bytes(rows, D, ctypes.byref(n)) == echo.ECHO_OK
    assert n.value == 304 * (16 + 2 * kept * (D + 2) * 4)
