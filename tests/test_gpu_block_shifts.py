"""4-bit rows that hold keys and values times powers of two: small ones survive, and what the
calls give back is as if no power had been there."""
import numpy as np
import pytest
import torch

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev
from test_gpu_block_attention import FP4, WIDE, Attn
from test_gpu_qk_norm_rope import Rope

pytestmark = pytest.mark.gpu


def test_small_groups_become_zeros_at_the_stated_border():
    """A group whose largest entry is 6 * 2^-10 or less becomes zeros; the next bf16 number does
    not. Largest entries of 2688 and more come back as at most 2688."""
    r = Rope(4, 1, 1, 128, 16, False, FP4, 16, norm=False, seed=1, max_pos=2)
    edge = 6 * 2.0 ** -10
    v = np.zeros((4, 1, 128))
    v[0], v[1], v[2], v[3] = edge, edge + 2.0 ** -15, 2688.0, 2704.0
    v[0, 0, ::2] *= -0.5
    r.v = dev(ref.bf16_bits(v).view(np.int16).reshape(v.shape)).view(torch.bfloat16)
    assert np.array_equal(r.v.double().cpu().numpy(), v)
    r.pos.zero_()
    r.pos_np[:] = 0
    echo.echo_qk_norm_rope(r.args())
    torch.cuda.synchronize()
    got = r.vo.double().cpu().numpy()
    assert (got[0] == 0).all() and (got[1] != 0).all() and (got[2:] == 2688).all()


@pytest.mark.parametrize("D,inter,T", [(128, False, 45), (64, True, 300), (64, False, 4)])
@pytest.mark.parametrize("scale,k_shift,v_shift", [(1e-4, 12, 9), (3000.0, -5, -3), (1.0, 0, 4), (1e-9, 32, 29)])
def test_rows_hold_the_entries_times_their_power(D, inter, T, scale, k_shift, v_shift):
    r = Rope(T, 4, 3, D, 32, inter, FP4, 16, norm=False, seed=T, scale=scale)
    echo.echo_qk_norm_rope(r.args(k_shift=k_shift, v_shift=v_shift))
    k2 = torch.empty_like(r.ko)
    echo.echo_qk_norm_rope(r.args(slot_map=None, rows=None, fmt=echo.BLOCK_BF16, k_out=k2, v_out=None))
    torch.cuda.synchronize()
    k, v = k2.double().cpu().numpy(), r.v.double().cpu().numpy()
    want = r.rows_np.copy()
    for t in range(T):
        blk, off = divmod(int(r.slot_np[t]), 16)
        for h in range(3):
            ks, vs = ref.write_token(want[blk * 3 + h], FP4, 16, D, off, k[t, h] * 2.0 ** k_shift, v[t, h] * 2.0 ** v_shift)
            assert np.array_equal(r.ko[t, h].double().cpu().numpy(), ks * 2.0 ** -k_shift)
            assert np.array_equal(r.vo[t, h].double().cpu().numpy(), vs * 2.0 ** -v_shift)
            # every group of 16 is kept (4 bits: half a step of the coarsest codes and of the scale)
            far = np.abs(v[t, h].reshape(-1, 16)).max(1) * (1 / 6 + 1 / 8)
            assert (np.abs(vs * 2.0 ** -v_shift - v[t, h]).reshape(-1, 16).max(1) <= far).all()
    got = r.rows.cpu().numpy().view(np.uint8).reshape(want.shape)
    assert np.array_equal(r.no_negative_zero(got), r.no_negative_zero(want)) and int(r.status) == 0
    r.check_heads(r.qo, r.q, None, np.ones(T, bool))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,cap", [([40, 700], None), ([900, 0, 2300], WIDE // 64), ([30] * 170, None)])
@pytest.mark.parametrize("k_shift,v_shift", [(3, -2), (-4, 32)])
def test_attention_takes_the_powers_back(D, lens, cap, k_shift, v_shift):
    a = Attn(FP4, D, 16, 8, 1, 2, lens, seed=2, cap=cap)
    a.kv = {at: (k * 2.0 ** -k_shift, v * 2.0 ** -v_shift) for at, (k, v) in a.kv.items()}
    args = a.args()
    args.k_shift, args.v_shift = k_shift, v_shift
    echo.echo_block_attention(args)
    a.check()


def test_small_keys_and_values_from_projection_to_output():
    """Values of about 2^-10, all of which would be lost without their power of two: written by
    the one call, attended over by the other."""
    T, H, Hk, D, bs = 200, 8, 2, 128, 16
    r = Rope(T, H, Hk, D, 64, False, FP4, bs, norm=False, seed=7, scale=2.0 ** -10)
    slot = np.random.default_rng(3).permutation(-(-T // bs))[np.arange(T) // bs] * bs + np.arange(T) % bs
    echo.echo_qk_norm_rope(r.args(slot_map=dev(slot.astype(np.int32)), k_shift=10, v_shift=11))
    a = Attn(FP4, D, bs, H, Hk, 1, [T], seed=1)
    a.table[0] = slot[::bs] // bs
    a.kv = {(a.row(0, h, p // bs), p % bs): (r.ko[p, h].double().cpu().numpy(), r.vo[p, h].double().cpu().numpy())
            for p in range(T) for h in range(Hk)}
    a.rows_np = r.rows_np
    a.dev()
    a.rows.copy_(r.rows)
    echo.echo_block_attention(echo.make_block_attention_args(
        a.q, a.rows, a.t, a.ctx, Hk, a.scale, a.out, a.lse, a.ws, fmt=FP4, block_tokens=bs, dev_status=a.status,
        k_shift=10, v_shift=11))
    a.check()
    assert (a.out.float().abs().amax(-1) > 0).all()
