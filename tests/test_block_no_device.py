"""The block calls on a machine without a CUDA device: an error, not a signal.  The argument
blocks hold invalid pointers, so that these calls are made only where nothing can run."""
import os
import subprocess
import sys

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CALL = """
import ctypes, sys
sys.path[:0] = [{here!r}, {root!r}]
import sparse_attention_kv_fp8_gb300 as echo
import test_block_abi as abi
args = {{"echo_block_tables": abi.tables_args(), "echo_qk_norm_rope": abi.rope_args(slot_map=None),
        "echo_block_attention": abi.attn_args({kw})}}[{name!r}]
lib = echo.load_library()
print(getattr(lib, {name!r})(ctypes.byref(args), None), lib.echo_last_error_string().decode())
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="a device is there: invalid pointers would reach it")
@pytest.mark.parametrize("name,kw", [
    ("echo_block_tables", ""), ("echo_qk_norm_rope", ""), ("echo_block_attention", ""),
    ("echo_block_attention", "max_blocks=60000"), ("echo_block_attention", "B=1000, format=1"),
])
def test_an_error_without_a_device(name, kw):
    """In a process of its own: a signal there is a failure here."""
    code = CALL.format(here=HERE, root=os.path.dirname(HERE), name=name, kw=kw)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    status, why = r.stdout.split(" ", 1)
    assert int(status) == 2 and why.strip(), r.stdout       # ECHO_ECUDA, with its reason
