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
