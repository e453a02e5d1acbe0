"""Powers of two in 4-bit rows: what the calls refuse.  No GPU needed."""
import ctypes

import pytest

import sparse_attention_kv_fp8_gb300 as echo
from test_block_abi import attn_args, lib, rope_args  # noqa: F401


@pytest.mark.parametrize("bad,why", [
    (dict(k_shift=1), b"4-bit"), (dict(v_shift=-1), b"4-bit"), (dict(format=1, k_shift=33), b"[-32, 32]"),
    (dict(format=1, v_shift=-33), b"[-32, 32]"),
])
def test_refused_shifts(lib, bad, why):  # noqa: F811
    for call, args in ((lib.echo_qk_norm_rope, rope_args), (lib.echo_block_attention, attn_args)):
        assert call(ctypes.byref(args(**bad)), None) == echo.ECHO_EINVAL
        assert why in lib.echo_last_error_string(), lib.echo_last_error_string()


def test_a_scale_that_the_shift_takes_out_of_range(lib):  # noqa: F811
    assert lib.echo_block_attention(ctypes.byref(attn_args(format=1, k_shift=-32, scale=1e30)), None) == echo.ECHO_EINVAL
    assert b"2^-k_shift" in lib.echo_last_error_string()
