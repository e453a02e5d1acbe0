"""The block calls' C ABI and host-side refusals; the references the GPU tests compare
with, against hand-computed values.  No GPU needed."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo
from sparse_attention_kv_fp8_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return echo.load_library()


def test_block_struct_layouts_match_the_header():
    structs = {"echo_block_tables_args": echo.c_block_tables_args, "echo_qk_norm_rope_args": echo.c_qk_norm_rope_args,
               "echo_block_attention_args": echo.c_block_attention_args}
    body = "".join(f'printf("{n} %zu\\n", sizeof({n}));\n' + "".join(
        f'printf("{n}.{f[0]} %zu\\n", offsetof({n}, {f[0]}));\n' for f in c._fields_) for n, c in structs.items())
    prog = "#include <stdio.h>\n#include <stddef.h>\n#include \"echo.h\"\nint main(void) {\n" + body + "return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(c, "w").write(prog)
        subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        lines = dict(l.rsplit(" ", 1) for l in subprocess.check_output([exe], text=True).splitlines())
    for n, c in structs.items():
        assert int(lines[n]) == ctypes.sizeof(c), n
        for f in c._fields_:
            assert int(lines[f"{n}.{f[0]}"]) == getattr(c, f[0]).offset, (n, f[0])


def test_row_elems(lib):
    assert echo.block_row_elems(echo.BLOCK_BF16, 64, 128) == 2 * 64 * 128
    assert echo.block_row_elems(echo.BLOCK_FP4, 64, 128) == 4 * 18 * 128 // 2
    assert echo.block_row_elems(echo.BLOCK_FP4, 16, 64) == 18 * 64 // 2
    for bad in ((2, 64, 128), (0, 24, 128), (0, 0, 128), (0, -16, 64), (0, 64, 96), (0, 512, 128), (1, 1024, 128)):
        with pytest.raises(echo.EchoError):
            echo.block_row_elems(*bad)
    assert lib.echo_block_row_elems(0, 64, 128, None) == echo.ECHO_EINVAL


def tables_args(**kw):
    a = echo.c_block_tables_args(16, 32, 4, 64, 48, 64, 8, 32, 80, 96, 112, 128, 144, None, 16, 160)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,why", [
    (dict(B=-1), b"B must"), (dict(B=16385), b"B must"), (dict(block_tokens=0), b"positive"),
    (dict(max_blocks=0), b"positive"), (dict(n_blocks=0), b"positive"), (dict(max_new=-1), b"max_new"),
    (dict(max_new=(1 << 30) + 1), b"max_new"), (dict(max_blocks=1 << 26, block_tokens=64), b"below 2^31"),
    (dict(n_blocks=1 << 26, block_tokens=64), b"below 2^31"), (dict(free_count=None), b"NULL"),
    (dict(free_blocks=None), b"NULL"), (dict(old_len=None), b"NULL"), (dict(table=None), b"NULL"),
    (dict(slot_map=None), b"slot_map"), (dict(free_count_out=80), b"different"), (dict(len_out=16), b"len_out"),
    (dict(len_out=32), b"len_out"), (dict(B=1024, max_blocks=1 << 20, block_tokens=1), b"below 2^30"),
    (dict(n_blocks=1 << 30, block_tokens=1), b"below 2^30"),
])
def test_block_tables_refusals(lib, bad, why):
    assert lib.echo_block_tables(ctypes.byref(tables_args(**bad)), None) == echo.ECHO_EINVAL
    assert why in lib.echo_last_error_string(), lib.echo_last_error_string()


def rope_args(**kw):
    a = echo.c_qk_norm_rope_args()
    vals = dict(q=16, k=32, v=48, q_stride=2048, k_stride=512, v_stride=512, T=4, n_heads=16, n_kv_heads=4,
                head_dim=128, q_weight=None, k_weight=None, eps=1e-6, interleaved=0, cos_sin=64, max_pos=100,
                rope_dim=128, positions=80, q_out=96, k_out=None, v_out=None, slot_map=4, rows=None, n_rows=8,
                format=0, block_tokens=64, dev_status=None)
    for k, v in {**vals, **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,why", [
    (dict(T=-1), b"bad sizes"), (dict(n_heads=0), b"bad sizes"), (dict(n_kv_heads=0), b"bad sizes"),
    (dict(head_dim=96), b"head_dim"), (dict(rope_dim=8), b"rope_dim"), (dict(rope_dim=24), b"rope_dim"),
    (dict(rope_dim=144), b"rope_dim"), (dict(max_pos=0), b"max_pos"), (dict(eps=-1.0), b"eps"),
    (dict(eps=float("nan")), b"eps"), (dict(interleaved=2), b"interleaved"), (dict(format=2), b"format"),
    (dict(block_tokens=20), b"block_tokens"), (dict(q=None), b"NULL"), (dict(positions=None), b"NULL"),
    (dict(cos_sin=None), b"NULL"), (dict(q_out=None), b"NULL"), (dict(q=18), b"16-byte"), (dict(cos_sin=68), b"16-byte"),
    (dict(k_out=8), b"16-byte"), (dict(q_stride=2052), b"multiples of 8"), (dict(v_stride=1), b"multiples of 8"),
    (dict(q_out=16, q_stride=2056), b"one after another"), (dict(k_out=32, k_stride=2048), b"one after another"),
    (dict(v_out=48, v_stride=2048), b"one after another"),
    (dict(v=None), b"v is NULL"), (dict(), b"without rows"), (dict(rows=8), b"16-byte"), (dict(rows=16, n_rows=0), b"without rows"),
])
def test_qk_norm_rope_refusals(lib, bad, why):
    assert lib.echo_qk_norm_rope(ctypes.byref(rope_args(**bad)), None) == echo.ECHO_EINVAL
    assert why in lib.echo_last_error_string(), lib.echo_last_error_string()


def attn_args(**kw):
    a = echo.c_block_attention_args()
    vals = dict(q=16, rows=32, n_rows=8, format=0, block_tokens=64, head_dim=128, table=48, sel=None, table_heads=1,
                max_blocks=4, ctx_len=64, B=2, n_q=1, n_heads=32, n_kv_heads=8, sinks=0, window=0, scale=0.1, out=80,
                lse=None, workspace=256, workspace_bytes=1 << 30, dev_status=None)
    for k, v in {**vals, **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,why", [
    (dict(B=-1), b"bad sizes"), (dict(n_q=0), b"bad sizes"), (dict(n_q=65), b"bad sizes"), (dict(n_heads=12), b"multiple"),
    (dict(n_kv_heads=0), b"multiple"), (dict(n_q=64, n_heads=256, n_kv_heads=8), b"1024"), (dict(format=3), b"format"),
    (dict(block_tokens=40), b"block_tokens"), (dict(head_dim=80), b"head_dim"), (dict(table_heads=2), b"table_heads"),
    (dict(max_blocks=0), b"max_blocks"), (dict(max_blocks=1 << 25), b"max_blocks"), (dict(sinks=-1), b"sinks"),
    (dict(window=-4), b"sinks"), (dict(n_rows=0), b"n_rows"), (dict(scale=float("inf")), b"finite"),
    (dict(q=None), b"NULL"), (dict(rows=None), b"NULL"), (dict(table=None), b"NULL"), (dict(out=None), b"NULL"),
    (dict(workspace=None), b"NULL"), (dict(q=24), b"16-byte"), (dict(rows=8), b"16-byte"), (dict(workspace=128), b"256-byte"),
    (dict(workspace_bytes=100), b"smaller"), (dict(out=16), b"out must not"), (dict(B=1 << 30), b"too large"),
])
def test_block_attention_refusals(lib, bad, why):
    assert lib.echo_block_attention(ctypes.byref(attn_args(**bad)), None) == echo.ECHO_EINVAL
    assert why in lib.echo_last_error_string(), lib.echo_last_error_string()


def test_workspace_bytes(lib):
    n = ctypes.c_size_t()
    sizes = []
    for rows in (1, 8, 9, 16, 17, 32, 33, 1024):
        assert lib.echo_block_attention_workspace_bytes(rows, 128, ctypes.byref(n)) == echo.ECHO_OK
        sizes.append(n.value)
    assert sizes[0] == sizes[1] < sizes[2] == sizes[3] < sizes[4] == sizes[5] == sizes[6] == sizes[7]
    for rows, D in ((0, 128), (1025, 128), (8, 32)):
        assert lib.echo_block_attention_workspace_bytes(rows, D, ctypes.byref(n)) == echo.ECHO_EINVAL
    assert lib.echo_block_attention_workspace_bytes(8, 128, None) == echo.ECHO_EINVAL


def test_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(echo.EchoError, match="CUDA"):
        echo.make_block_tables_args(i, i, 64, i.view(4, 1), i, i[:1], i[1:2], i)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(echo.EchoError, match="CUDA"):
        echo.make_qk_norm_rope_args(q, q, q, i[:2], torch.zeros(8, 128), q)
    with pytest.raises(echo.EchoError, match="rows have"):
        echo.make_block_attention_args(q[:, None], torch.zeros(2, 8, dtype=torch.int16), i.view(2, 2), i[:2], 4, 0.1,
                                       q[:, None], None, None)


# ---- the references themselves -------------------------------------------------

def test_reference_quantisation_on_hand_values():
    x = np.zeros(16)
    x[:8] = [6.0, -3.0, 0.25, 0.26, 0.75, -5.0, 1.25, 2.5]     # amax 6: scale 1
    c, s = ref.quantise(x)
    assert ref.E4M3[s[0]] == 1.0
    # ties: 0.25 -> 0, 0.75 -> 1 (code 2), 5 -> 4 (code 6), 1.25 -> 1 (code 2), 2.5 -> 2 (code 4)
    assert list(c[:8]) == [7, 8 | 5, 0, 1, 2, 8 | 6, 2, 4]
    c, s = ref.quantise(np.full(16, 1e-4))                      # below half the smallest scale
    assert s[0] == 0 and not c.any()
    c, s = ref.quantise(np.full(16, 1e30))                      # saturates
    assert ref.E4M3[s[0]] == 448 and (c == 7).all()


def test_reference_layout_covers_every_byte_once():
    for fmt in (echo.BLOCK_BF16, echo.BLOCK_FP4):
        for D in (64, 128):
            for bs in (16, 48):
                seen = np.zeros(2 * echo.block_row_elems(fmt, bs, D), int)
                for off in range(bs):
                    for i in ref.token_bytes(fmt, bs, D, off):
                        seen[i] += 1
                assert (seen == 1).all()


def test_reference_tables_on_a_hand_case():
    # bs 4; request 0 shrinks 9 -> 2 (frees blocks 11, 12), request 1 grows 3 -> 5, request 2
    # starts with 4 tokens; the stack holds 20, 21
    table = np.array([[10, 11, 12], [13, -1, -1], [-1, -1, -1]], np.int32)
    free = np.array([20, 21, -1, -1, -1, -1], np.int32)
    t, f, n, slot, pos, cu, ln, ex = ref.block_tables([9, 3, 0], [2, 5, 4], 4, table, free, 2, 8)
    assert list(f[:4]) == [20, 21, 11, 12] and n == 2 and not ex
    assert t[1, 1] == 12 and t[2, 0] == 11
    assert list(slot) == [13 * 4 + 3, 12 * 4, 44, 45, 46, 47, -1, -1] and list(pos) == [3, 4, 0, 1, 2, 3, -1, -1]
    assert list(cu) == [0, 0, 2, 6] and list(ln) == [2, 5, 4]
    _, _, n, slot, _, _, ln, ex = ref.block_tables([0, 0, 0], [9, 1, 0], 4, table, free, 2, 10)
    assert ex and n == 2 and (slot == -1).all() and list(ln) == [0, 0, 0]   # 3 do not fit; nor does a later 1
