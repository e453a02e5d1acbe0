"""C ABI and host-side refusals of the block calls that select, weigh, evict and share; the
references of their GPU tests on hand values.  No GPU needed."""
import ctypes
import os
import subprocess
import sys
import tempfile

import numpy as np
import pytest
import torch

import block_ref as ref
import more_ref
import sparse_attention_kv_fp8_gb300 as echo
from sparse_attention_kv_fp8_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
STRUCTS = {"echo_block_summary_args": echo.c_block_summary_args, "echo_block_scores_args": echo.c_block_scores_args,
           "echo_block_select_args": echo.c_block_select_args, "echo_block_weights_args": echo.c_block_weights_args,
           "echo_block_evict_args": echo.c_block_evict_args, "echo_prefix_attention_args": echo.c_prefix_attention_args}


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return echo.load_library()


def test_struct_layouts_match_the_header():
    body = "".join(f'printf("{n} %zu\\n", sizeof({n}));\n' + "".join(
        f'printf("{n}.{f[0]} %zu\\n", offsetof({n}, {f[0]}));\n' for f in c._fields_) for n, c in STRUCTS.items())
    prog = "#include <stdio.h>\n#include <stddef.h>\n#include \"echo.h\"\nint main(void) {\n" + body + "return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(c, "w").write(prog)
        subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        lines = dict(l.rsplit(" ", 1) for l in subprocess.check_output([exe], text=True).splitlines())
    for n, c in STRUCTS.items():
        assert int(lines[n]) == ctypes.sizeof(c), n
        for f in c._fields_:
            assert int(lines[f"{n}.{f[0]}"]) == getattr(c, f[0]).offset, (n, f[0])


def block(cls, base, **kw):
    a = cls()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


ROWS = dict(rows=32, n_rows=8, format=0, block_tokens=64, head_dim=128)
TABLE = dict(table=48, table_heads=1, max_blocks=4)
HEADS = dict(B=2, n_q=1, n_heads=32, n_kv_heads=8, scale=0.1)
BASE = {
    "echo_block_summary": (echo.c_block_summary_args, {**ROWS, **TABLE, **dict(old_len=None, new_len=64, B=2, n_kv_heads=8, summary=80)}),
    "echo_block_scores": (echo.c_block_scores_args, {**TABLE, **HEADS, **dict(q=16, summary=32, n_rows=8, block_tokens=64, head_dim=128,
                                                                             ctx_len=64, scores=80)}),
    "echo_block_select": (echo.c_block_select_args, {**TABLE, **dict(scores=16, ctx_len=32, B=2, n_q=1, n_kv_heads=8, block_tokens=64,
                                                                    k=4, first=1, last=1, sel=64, sel_rows=80, len_out=96)}),
    "echo_block_weights": (echo.c_block_weights_args, {**ROWS, **TABLE, **HEADS, **dict(q=16, ctx_len=64, old_len=80, lse=96, acc=112,
                                                                                       acc_out=128, decay=1.0)}),
    "echo_block_evict": (echo.c_block_evict_args, {**ROWS, **TABLE, **dict(len=64, len_out=80, B=2, n_kv_heads=8, keep=100, sinks=4,
                                                                          recent=32, acc=96, acc_out=112, pos=128, pos_out=144,
                                                                          pos_len=160, next_pos=176, workspace=256,
                                                                          workspace_bytes=1 << 30)}),
    "echo_prefix_attention": (echo.c_prefix_attention_args, {**ROWS, **TABLE, **HEADS, **dict(
        q=16, prefix_table=64, prefix_len=80, group_start=96, n_groups=2, prefix_heads=1, max_prefix_blocks=8, ctx_len=112, out=128,
        lse=None, workspace=256, workspace_bytes=1 << 40)}),
}


def make(name, **kw):
    return block(*BASE[name], **kw)


BIG = 1 << 30
CASES = [
    *[(n, d, w) for n in ("echo_block_summary", "echo_block_weights", "echo_block_evict", "echo_prefix_attention") for d, w in [
        (dict(format=2), b"format"), (dict(block_tokens=24), b"block_tokens"), (dict(head_dim=96), b"head_dim"),
        (dict(n_rows=0), b"n_rows"), (dict(rows=None), b"NULL"), (dict(rows=8), b"16-byte"), (dict(B=-1), b"B"),
        (dict(block_tokens=512), b"65536")]],
    *[(n, d, w) for n in BASE for d, w in [
        (dict(table_heads=3), b"table_heads"), (dict(max_blocks=0), b"max_blocks"), (dict(max_blocks=BIG), b"max_blocks")]],
    *[(n, dict(n_kv_heads=0), b"n_kv_heads") for n in ("echo_block_summary", "echo_block_select", "echo_block_evict")],
    *[(n, d, w) for n in ("echo_block_scores", "echo_block_weights", "echo_prefix_attention") for d, w in [
        (dict(n_heads=12), b"multiple"), (dict(n_q=0), b"bad sizes"), (dict(scale=float("nan")), b"finite"), (dict(q=24), b"16-byte"),
        (dict(q=None), b"NULL"), (dict(B=1 << 28, n_heads=64), b"too large")]],
    ("echo_block_summary", dict(B=16385), b"B must"), ("echo_block_summary", dict(table=None), b"NULL"),
    ("echo_block_summary", dict(new_len=None), b"NULL"), ("echo_block_summary", dict(summary=None), b"NULL"),
    ("echo_block_summary", dict(summary=72), b"16-byte"), ("echo_block_summary", dict(k_shift=1), b"4-bit"),
    ("echo_block_summary", dict(format=1, k_shift=33), b"[-32, 32]"),
    ("echo_block_summary", dict(B=16384, max_blocks=1 << 17, block_tokens=16), b"2^30"),
    ("echo_block_scores", dict(head_dim=32), b"head_dim"), ("echo_block_scores", dict(summary=None), b"NULL"),
    ("echo_block_scores", dict(scores=None), b"NULL"), ("echo_block_scores", dict(n_rows=0), b"n_rows"),
    ("echo_block_scores", dict(B=65536, max_blocks=1 << 20, block_tokens=16, n_heads=8), b"2^31"),
    ("echo_block_scores", dict(B=1, n_q=65536, n_heads=16384, n_kv_heads=1, table_heads=1), b"2^30"),
    ("echo_block_select", dict(k=0), b"k must"), ("echo_block_select", dict(first=-1), b"first"), ("echo_block_select", dict(last=4), b"first"),
    ("echo_block_select", dict(max_blocks=32769), b"32768"), ("echo_block_select", dict(table=None), b"sel_rows"),
    ("echo_block_select", dict(scores=None), b"NULL"), ("echo_block_select", dict(sel=None), b"NULL"),
    ("echo_block_select", dict(len_out=32), b"len_out"), ("echo_block_select", dict(B=BIG), b"too large"),
    ("echo_block_select", dict(n_q=0), b"bad sizes"),
    ("echo_block_weights", dict(n_q=300), b"1024"), ("echo_block_weights", dict(decay=float("inf")), b"finite"),
    ("echo_block_weights", dict(lse=None), b"NULL"), ("echo_block_weights", dict(acc_out=None), b"NULL"),
    ("echo_block_weights", dict(acc=None), b"old_len needs acc"), ("echo_block_weights", dict(format=1, k_shift=-32, scale=1e30), b"2^-k_shift"),
    ("echo_block_weights", dict(B=1 << 22, n_heads=8, max_blocks=1 << 20, block_tokens=64), b"2^31"),
    ("echo_block_evict", dict(keep=0), b"keep"), ("echo_block_evict", dict(sinks=69), b"sum at most keep"),
    ("echo_block_evict", dict(sinks=-1), b"sinks"), ("echo_block_evict", dict(pos=None), b"go together"),
    ("echo_block_evict", dict(next_pos=None), b"go together"),
    ("echo_block_evict", dict(pos=None, pos_out=None, pos_len=None, next_pos=None), b"recent needs pos"),
    ("echo_block_evict", dict(len_out=64), b"len_out"), ("echo_block_evict", dict(len_out=160), b"len_out"),
    ("echo_block_evict", dict(acc=None), b"NULL"), ("echo_block_evict", dict(workspace=None), b"NULL"),
    *[("echo_block_evict", {f: 72}, b"16-byte") for f in ("acc", "acc_out", "pos", "pos_out")],
    ("echo_block_evict", dict(workspace=128), b"256-byte"), ("echo_block_evict", dict(workspace_bytes=100), b"smaller"),
    ("echo_block_evict", dict(B=1 << 23), b"2^26"),
    ("echo_prefix_attention", dict(n_groups=0), b"n_groups"), ("echo_prefix_attention", dict(n_groups=65537), b"n_groups"),
    ("echo_prefix_attention", dict(prefix_heads=2), b"prefix_heads"), ("echo_prefix_attention", dict(max_prefix_blocks=0), b"max_prefix_blocks"),
    ("echo_prefix_attention", dict(n_groups=65536, max_prefix_blocks=4096), b"n_groups * n_kv_heads"),
    ("echo_prefix_attention", dict(prefix_table=None), b"NULL"),
    ("echo_prefix_attention", dict(prefix_len=None), b"NULL"), ("echo_prefix_attention", dict(group_start=None), b"NULL"),
    ("echo_prefix_attention", dict(ctx_len=None), b"go together"), ("echo_prefix_attention", dict(out=None), b"NULL"),
    ("echo_prefix_attention", dict(out=16), b"out must not"), ("echo_prefix_attention", dict(workspace=64), b"256-byte"),
    ("echo_prefix_attention", dict(workspace_bytes=1000), b"smaller"), ("echo_prefix_attention", dict(n_q=65), b"bad sizes"),
    ("echo_prefix_attention", dict(n_rows=BIG + 1), b"n_rows"), ("echo_prefix_attention", dict(k_shift=1), b"4-bit"),
    ("echo_prefix_attention", dict(B=1 << 20, max_prefix_blocks=1 << 24), b"prefixes too large"),
]


@pytest.mark.parametrize("name,bad,why", CASES)
def test_refusals(lib, name, bad, why):
    assert getattr(lib, name)(ctypes.byref(make(name, **bad)), None) == echo.ECHO_EINVAL
    assert why in lib.echo_last_error_string(), lib.echo_last_error_string()


@pytest.mark.parametrize("name", list(BASE))
def test_no_arguments_and_no_requests(lib, name):
    assert getattr(lib, name)(None, None) == echo.ECHO_EINVAL
    assert getattr(lib, name)(ctypes.byref(make(name, B=0)), None) == echo.ECHO_OK


def test_workspace_sizes(lib):
    n = ctypes.c_size_t()
    assert lib.echo_block_evict_workspace_bytes(2, 8, 100, ctypes.byref(n)) == echo.ECHO_OK
    assert n.value == 256 + 2 * 8 * 100 * 8           # a count each (rounded up), (from, to) of up to `keep` moves
    assert lib.echo_block_evict_workspace_bytes(2, 8, 0, ctypes.byref(n)) == echo.ECHO_EINVAL
    assert lib.echo_block_evict_workspace_bytes(2, 8, 100, None) == echo.ECHO_EINVAL
    assert lib.echo_prefix_attention_workspace_bytes(64, 1, 64, 8, 128, ctypes.byref(n)) == echo.ECHO_OK
    # at least the parts of each row, fp32, twice, and a slot of 256 rows for each of 160 CTAs
    assert n.value >= 2 * 64 * 64 * 128 * 4 + 160 * 256 * 128 * 4
    for bad in ((64, 1, 64, 7, 128), (64, 1, 64, 8, 96), (-1, 1, 64, 8, 128), (1, 1025, 8, 8, 128)):
        assert lib.echo_prefix_attention_workspace_bytes(*bad, ctypes.byref(n)) == echo.ECHO_EINVAL
    assert lib.echo_prefix_attention_workspace_bytes(1, 1, 8, 8, 128, None) == echo.ECHO_EINVAL


def test_version(lib):
    assert echo.version() & 0xFFFF >= 8


CALL = """
import ctypes, sys
sys.path[:0] = [{here!r}, {root!r}]
import sparse_attention_kv_fp8_gb300 as echo
import test_more_block_abi as abi
lib = echo.load_library()
print(getattr(lib, {name!r})(ctypes.byref(abi.make({name!r})), None), lib.echo_last_error_string().decode())
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="a device is there: invalid pointers would reach it")
@pytest.mark.parametrize("name", list(BASE))
def test_an_error_without_a_device(lib, name):
    """In a process of its own: a signal there is a failure here."""
    r = subprocess.run([sys.executable, "-c", CALL.format(here=HERE, root=ROOT, name=name)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    status, why = r.stdout.split(" ", 1)
    assert int(status) == 2 and why.strip(), r.stdout       # ECHO_ECUDA, with its reason


def test_references_on_hand_values():
    s = np.array([1.0, 5.0, np.nan, 5.0, -np.inf, 2.0])
    assert more_ref.select(s, 6, 2, 0, 0, [True] * 6) == [1, 3]
    assert more_ref.select(s, 6, 3, 1, 1, [True] * 6) == [0, 1, 5]
    assert more_ref.select(s, 4, 3, 0, 0, [True, False, True, True]) == [0, 2, 3]
    assert more_ref.select(s, 2, 4, 0, 0, [True] * 6) == [0, 1, -1, -1]
    acc = np.array([0.0, 3.0, 1.0, 0.0, 2.0, 5.0])
    assert list(more_ref.evict(acc, None, 6, 3, 0, 0, 0)) == [4, 1, 5]
    assert list(more_ref.evict(acc, None, 6, 3, 1, 0, 0)) == [0, 1, 5]
    assert list(more_ref.evict(acc, np.arange(6), 6, 3, 0, 2, 6)) == [4, 1, 5]
    assert list(more_ref.evict(acc, np.array([9, 0, 1, 2, 3, 4]), 6, 2, 0, 1, 10)) == [0, 5]
    assert list(more_ref.evict(acc, None, 2, 3, 0, 0, 0)) == [0, 1]


@pytest.mark.parametrize("fmt", [echo.BLOCK_BF16, echo.BLOCK_FP4])
def test_packed_rows_agree_with_written_tokens(fmt):
    g = np.random.default_rng(3)
    bs, D = 32, 64
    k, v = (ref.bf16_round(g.standard_normal((2, bs, D))) for _ in range(2))
    rows, kv, vv = more_ref.pack_rows(fmt, bs, D, k, v)
    for r in range(2):
        want = np.zeros_like(rows[0])
        for t in range(bs):
            a, b = ref.write_token(want, fmt, bs, D, t, k[r, t], v[r, t])
            assert (a == kv[r, t]).all() and (b == vv[r, t]).all()
        assert (rows[r] == want).all()
