"""Sizes and numbers that the block calls which select, weigh, evict and share refuse, beside those of
test_more_block_abi.py.  No GPU needed."""
import ctypes

import sparse_attention_kv_fp8_gb300 as echo
from test_more_block_abi import lib, make  # noqa: F401


def refused(lib, name, why, **bad):  # noqa: F811
    assert getattr(lib, name)(ctypes.byref(make(name, **bad)), None) == echo.ECHO_EINVAL
    assert why in lib.echo_last_error_string(), lib.echo_last_error_string()


def test_selection_refuses_a_negative_number_of_rows(lib):  # noqa: F811
    refused(lib, "echo_block_select", b"n_rows", n_rows=-1)


def test_eviction_refuses_slots_that_its_steps_cannot_count(lib):  # noqa: F811
    """A step of 16384 slots from one below 2^31 - 1024 would pass 31 bits and be read."""
    for slots in ((1 << 31) - 1024, (1 << 31) - (1 << 14), (1 << 31) - (1 << 16) + 16):
        refused(lib, "echo_block_evict", b"2^31 - 2^16", block_tokens=16, max_blocks=slots // 16)
    a = make("echo_block_evict", B=0, block_tokens=16, max_blocks=((1 << 31) - (1 << 16)) // 16)
    assert lib.echo_block_evict(ctypes.byref(a), None) == echo.ECHO_OK
