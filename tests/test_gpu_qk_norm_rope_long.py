"""echo_qk_norm_rope at sizes whose warps take long runs of heads (16 of the queries, 8 of the
keys and values, cut short by odd head counts): against the formulas in 64 bits, all rows."""
import numpy as np
import pytest
import torch

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev
from test_gpu_qk_norm_rope import BF16, FP4, Rope

pytestmark = pytest.mark.gpu
# heads, KV heads, tokens by format
HEADS = {128: (35, 11, {BF16: 5803, FP4: 2401}), 64: (70, 9, {BF16: 7501, FP4: 3003})}


def long_call(fmt, D, inter, **kw):
    Hq, Hk, T = HEADS[D]
    # the rule of the launcher: at least 8 KV heads, and warps, at one head each, past a threshold
    warps = -(-T[fmt] // (256 // D)) * (Hq + 2 * Hk)
    assert Hk >= 8 and warps > (65536 if fmt == FP4 else 163840)
    return Rope(T[fmt], Hq, Hk, D, D, inter, fmt, 64, seed=D + fmt, **kw)


def want_rows(r, k, v):
    """The cache rows after the call: the tokens of one place in their blocks at a time."""
    want = r.rows_np.copy()
    for off in range(r.bs):
        t = np.nonzero(r.slot_np % r.bs == off)[0]
        row = (r.slot_np[t] // r.bs)[:, None] * r.Hk + np.arange(r.Hk)
        at = ref.token_bytes(r.fmt, r.bs, r.D, off)
        if r.fmt == BF16:
            parts = [ref.bf16_bits(x[t]).reshape(t.size, r.Hk, 2 * r.D) for x in (k, v)]
        else:
            pack = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)
            (kc, ks), (vc, vs) = ref.quantise(k[t]), ref.quantise(v[t])
            parts = [pack(kc), ks, pack(vc), vs]
        for i, p in zip(at, parts):
            want[row[..., None], i] = p
    return want


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D", [128, 64])
def test_long_runs_of_heads(fmt, D, inter):
    r = long_call(fmt, D, inter)
    echo.echo_qk_norm_rope(r.args())
    torch.cuda.synchronize()
    live = np.ones(r.T, bool)
    r.check_heads(r.qo, r.q, r.wq, live)
    k2 = r.ko
    if fmt == FP4:               # the keys before quantisation: a bf16 call gives them
        k2 = torch.empty_like(r.ko)
        echo.echo_qk_norm_rope(r.args(slot_map=None, rows=None, fmt=BF16, k_out=k2, v_out=None))
    r.check_heads(k2, r.k, r.wk, live)
    k, v = k2.double().cpu().numpy(), r.v.double().cpu().numpy()
    kv, vv = (k, v) if fmt == BF16 else (ref.code_values(*ref.quantise(x)) for x in (k, v))
    assert np.array_equal(r.ko.double().cpu().numpy(), kv) and np.array_equal(r.vo.double().cpu().numpy(), vv)
    got, want = r.rows.cpu().numpy().view(np.uint8).reshape(r.rows_np.shape), want_rows(r, k, v)
    if fmt == FP4:               # a zero code may carry either sign
        got, want = r.no_negative_zero(got), r.no_negative_zero(want)
    assert np.array_equal(got, want) and int(r.status) == 0


@pytest.mark.parametrize("fmt,D,inter", [(BF16, 128, False), (FP4, 128, True), (BF16, 64, True), (FP4, 64, False)])
def test_long_runs_of_heads_in_place(fmt, D, inter):
    r = long_call(fmt, D, inter, fused=False)
    echo.echo_qk_norm_rope(r.args())
    rows = r.rows.clone()
    r.rows.copy_(dev(r.rows_np.view(np.int16)))
    echo.echo_qk_norm_rope(echo.make_qk_norm_rope_args(r.q, r.k, r.v, r.pos, r.cs, r.q, r.wq, r.wk, 1e-5, inter, r.slot,
                                                       r.rows, fmt, 64, k_out=r.k, v_out=r.v, dev_status=r.status))
    torch.cuda.synchronize()
    for got, want in ((r.q, r.qo), (r.k, r.ko), (r.v, r.vo), (r.rows, rows)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert int(r.status) == 0
