"""echo_qk_norm_rope on the GPU against the formulas in 64 bits, and its cache rows, byte by
byte, against the layouts' definition."""
import numpy as np
import pytest
import torch

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev, pinned_host_pool

pytestmark = pytest.mark.gpu
BF16, FP4 = echo.BLOCK_BF16, echo.BLOCK_FP4


class Rope:
    def __init__(self, T, Hq, Hk, D, rd, inter, fmt, bs, norm=True, seed=0, fused=True, max_pos=5000, scale=1.0, host=False):
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        c = np.random.default_rng(seed)
        self.__dict__.update(T=T, Hq=Hq, Hk=Hk, D=D, rd=rd, inter=inter, fmt=fmt, bs=bs)
        pad = 8 if fused else 0
        x = (torch.randn(T, (Hq + 2 * Hk) * D + pad, generator=g, device="cuda") * scale).bfloat16()
        cut = lambda a, n: x[:, a * D:(a + n) * D].unflatten(1, (n, D))
        self.q, self.k, self.v = cut(0, Hq), cut(Hq, Hk), cut(Hq + Hk, Hk)
        if not fused:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        self.wq = 1 + 0.2 * torch.randn(D, generator=g, device="cuda") if norm else None
        self.wk = 1 + 0.2 * torch.randn(D, generator=g, device="cuda") if norm else None
        self.cs = echo.rope_table(max_pos, rd)
        self.pos_np = c.integers(0, max_pos, T).astype(np.int32)
        n_blk = -(-T // bs) + 2
        self.slot_np = c.permutation(n_blk * bs)[:T].astype(np.int32)
        self.pos, self.slot = dev(self.pos_np), dev(self.slot_np)
        R = echo.block_row_elems(fmt, bs, D)
        self.rows_np = c.integers(0, 256, (n_blk * Hk, 2 * R)).astype(np.uint8)
        rows16 = self.rows_np.view(np.int16)
        self.rows = pinned_host_pool(rows16.view(np.uint16)) if host else dev(rows16)
        e = lambda *n: torch.full(n, 7.0, dtype=torch.bfloat16, device="cuda")
        self.qo, self.ko, self.vo = e(T, Hq, D), e(T, Hk, D), e(T, Hk, D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self, **kw):
        a = dict(q_weight=self.wq, k_weight=self.wk, eps=1e-5, interleaved=self.inter, slot_map=self.slot, rows=self.rows,
                 fmt=self.fmt, block_tokens=self.bs, k_out=self.ko, v_out=self.vo, dev_status=self.status)
        return echo.make_qk_norm_rope_args(self.q, self.k, self.v, self.pos, self.cs, self.qo, **{**a, **kw})

    def want(self, x, w):
        f = lambda t: None if t is None else t.double().cpu().numpy()
        pos = np.clip(self.pos_np, 0, self.cs.shape[0] - 1)
        return ref.norm_rope(f(x), f(w), 1e-5, f(self.cs)[pos], self.rd, self.inter)

    def check_heads(self, got, x, w, live):
        """A norm's mean adds D squares as a tree and is off by about 12 roundings of 2^-24,
        the rotation by 3 more: far under 2^-18 of |a cos| + |b sin|.  Then one rounding to bf16."""
        y, mag = self.want(x, w)
        d = np.abs(got.double().cpu().numpy() - y)
        far = 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * mag
        assert (d[live] <= far[live]).all(), (d[live] - far[live]).max()

    def check(self, status=0, rows=None):
        torch.cuda.synchronize()
        live = (self.pos_np >= 0) & (self.pos_np < self.cs.shape[0])
        self.check_heads(self.qo, self.q, self.wq, live)
        assert bool((self.qo[torch.from_numpy(~live).cuda()] == 7.0).all())
        assert int(self.status) == status
        v = self.v.double().cpu().numpy()
        if self.fmt == BF16:
            self.check_heads(self.ko, self.k, self.wk, live)
            k = self.ko.double().cpu().numpy()
            kv, vv = k, v
            assert np.array_equal(self.vo.double().cpu().numpy()[live], v[live])
        else:
            # the same arithmetic before quantisation: a bf16 call gives the keys
            k2 = torch.empty_like(self.ko)
            echo.echo_qk_norm_rope(self.args(slot_map=None, rows=None, fmt=BF16, k_out=k2, v_out=None, dev_status=None))
            self.check_heads(k2, self.k, self.wk, live)
            k = k2.double().cpu().numpy()
            kv, vv = ref.code_values(*ref.quantise(k)), ref.code_values(*ref.quantise(v))
            assert np.array_equal(self.ko.double().cpu().numpy()[live], kv[live])
            assert np.array_equal(self.vo.double().cpu().numpy()[live], vv[live])
        got = (self.rows if rows is None else rows).cpu().numpy().view(np.uint8).reshape(self.rows_np.shape)
        want = self.rows_np.copy()
        n_rows = want.shape[0]
        for t in np.nonzero(live & (self.slot_np >= 0))[0]:
            blk, off = divmod(int(self.slot_np[t]), self.bs)
            for h in range(self.Hk):
                if blk * self.Hk + h < n_rows:
                    ref.write_token(want[blk * self.Hk + h], self.fmt, self.bs, self.D, off, k[t, h], v[t, h])
        if self.fmt == FP4:      # a zero code may carry either sign
            got, want = self.no_negative_zero(got), self.no_negative_zero(want)
        assert np.array_equal(got, want)

    def no_negative_zero(self, rows):
        x = rows.reshape(-1, 18 * self.D).copy()
        c = x[:, :16 * self.D]
        lo, hi = c & 15, c >> 4
        x[:, :16 * self.D] = np.where(lo == 8, 0, lo) | (np.where(hi == 8, 0, hi) << 4)
        return x


CASES = [
    (1, 64, 8, 128, 128, False), (1, 1, 1, 64, 64, True), (2, 6, 2, 64, 32, False), (3, 5, 5, 128, 16, True),
    (7, 8, 1, 128, 64, False), (33, 7, 3, 64, 16, False), (130, 32, 8, 128, 128, True), (300, 64, 8, 128, 96, False),
    (500, 40, 8, 64, 48, True), (2001, 18, 3, 128, 128, False), (700, 5, 4, 64, 32, True),
]


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("T,Hq,Hk,D,rd,inter", CASES)
def test_norm_rope_and_cache(T, Hq, Hk, D, rd, inter, fmt):
    r = Rope(T, Hq, Hk, D, rd, inter, fmt, bs=[16, 64, 48][T % 3], seed=T, norm=T % 2 == 1, fused=T != 7)
    echo.echo_qk_norm_rope(r.args())
    r.check()


@pytest.mark.parametrize("fmt,D,inter", [(BF16, 128, False), (FP4, 128, True), (FP4, 64, False), (BF16, 64, True)])
def test_a_long_chunk(fmt, D, inter):
    """Enough heads for the longest runs per warp (16 and 8, cut short by the head counts)."""
    r = Rope(9001, 35 if D == 128 else 70, 2 if D == 128 else 5, D, D, inter, fmt, 64, seed=2)
    echo.echo_qk_norm_rope(r.args())
    r.check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_padding_bad_positions_and_unwritten_tokens(fmt):
    r = Rope(20, 4, 2, 128, 64, False, fmt, 16, seed=3)
    r.pos_np[[2, 5]] = -1                       # padding: nothing of the token is written
    r.pos_np[7] = 5000                          # past the table: left out and flagged
    r.slot_np[[1, 19]] = -1                     # no cache slot: q only
    r.slot_np[4] = (r.rows.shape[0] // 2) * 16 + 3   # a block past the rows: flagged
    r.pos.copy_(dev(r.pos_np)), r.slot.copy_(dev(r.slot_np))
    echo.echo_qk_norm_rope(r.args())
    r.check(echo.DEV_BAD_INDEX)
    keep = torch.from_numpy(np.isin(np.arange(20), [2, 5, 7])).cuda()
    assert bool((r.ko[keep] == 7.0).all()) and bool((r.vo[keep] == 7.0).all())


@pytest.mark.parametrize("scale", [1e-5, 1e-3, 100.0, 3000.0])
def test_values_near_the_ends_of_the_4_bit_range(scale):
    r = Rope(40, 2, 2, 128, 32, False, FP4, 16, norm=False, seed=11, scale=scale)
    echo.echo_qk_norm_rope(r.args())
    r.check()


def test_every_tie_of_the_4_bit_grid_goes_to_the_even_code():
    """Values on the borders between codes (and one bf16 step to either side), for every
    e4m3 scale a group maximum of 6 s gives."""
    r = Rope(126, 1, 1, 128, 16, False, FP4, 16, norm=False, seed=1, max_pos=2)
    edges = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    v = np.zeros((126, 8, 16))
    for i in range(126):                         # scale bytes 1 .. 126
        s = ref.E4M3[i + 1]
        e = edges * s
        up = ref.bf16_round(e * (1 + 2.0 ** -7))
        down = ref.bf16_round(e * (1 - 2.0 ** -8))
        v[i, 0, :7], v[i, 1, :7], v[i, 2, :7] = e, up, down
        v[i, 3, :7], v[i, 4, :7] = -e, -up
        v[i, 5, :8] = ref.GRID * s
        v[i, :, 15] = 6 * s
    r.v = dev(ref.bf16_bits(v.reshape(126, 1, 128)).view(np.int16).reshape(126, 1, 128)).view(torch.bfloat16)
    assert np.array_equal(r.v.double().cpu().numpy().reshape(v.shape), v)      # all exact in bf16
    echo.echo_qk_norm_rope(r.args())
    r.check()


def test_no_cache_no_values_and_in_place_queries():
    r = Rope(50, 8, 2, 128, 128, False, BF16, 16, seed=5, fused=False)
    q0 = r.q.clone()
    a = echo.make_qk_norm_rope_args(r.q, r.k, None, r.pos, r.cs, r.q, q_weight=r.wq, eps=1e-5)
    echo.echo_qk_norm_rope(a)
    torch.cuda.synchronize()
    r.qo, r.q = r.q, q0
    r.check_heads(r.qo, r.q, r.wq, np.ones(50, bool))


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("T,inter", [(5, True), (301, False), (14000, False)])
def test_queries_keys_and_values_in_place(T, inter, fmt):
    r = Rope(T, 16, 4, 128, 64, inter, fmt, 32, fused=False)
    echo.echo_qk_norm_rope(r.args())
    rows = r.rows.clone()
    r.rows.copy_(dev(r.rows_np.view(np.int16)))
    a = echo.make_qk_norm_rope_args(r.q, r.k, r.v, r.pos, r.cs, r.q, r.wq, r.wk, 1e-5, inter, r.slot, r.rows, fmt, 32,
                                    k_out=r.k, v_out=r.v, dev_status=r.status)
    echo.echo_qk_norm_rope(a)
    torch.cuda.synchronize()
    for got, want in ((r.q, r.qo), (r.k, r.ko), (r.v, r.vo), (r.rows, rows)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert int(r.status) == 0


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_rows_in_the_pinned_host_pool(fmt):
    r = Rope(60, 4, 2, 128, 128, False, fmt, 64, seed=6, host=True)
    echo.echo_qk_norm_rope(r.args())
    r.check()


def test_empty_call_and_refused_views():
    r = Rope(4, 4, 2, 128, 128, False, BF16, 16)
    e = lambda t: t[:0]
    echo.echo_qk_norm_rope(echo.make_qk_norm_rope_args(e(r.q), e(r.k), e(r.v), e(r.pos), r.cs, e(r.qo)))
    with pytest.raises(echo.EchoError, match="contiguous heads"):
        echo.make_qk_norm_rope_args(r.q[:, ::2], r.k, r.v, r.pos, r.cs, r.qo[:, ::2].contiguous())
    with pytest.raises(echo.EchoError, match="rows have"):
        r.args(block_tokens=32)
    with pytest.raises(echo.EchoError, match="one of"):
        r.args(q_weight=r.wq.half())


def test_large_rows_offsets_pass_32_bits():
    """Slots near the end of 5 GB of rows."""
    T, Hk, D, bs = 10, 2, 128, 64
    n_rows = 5 * (1 << 30) // (4 * bs * D)
    r = Rope(T, 4, Hk, D, 64, True, BF16, bs, seed=8)
    big = torch.empty(n_rows, 2 * bs * D, dtype=torch.int16, device="cuda")
    tail = r.rows.shape[0]
    assert n_rows % Hk == 0 and tail % Hk == 0
    big[-tail:].copy_(r.rows)
    slot = dev(r.slot_np + ((n_rows - tail) // Hk) * bs)
    echo.echo_qk_norm_rope(r.args(slot_map=slot, rows=big))
    r.check(rows=big[-tail:])


def test_captured_on_a_side_stream():
    r = Rope(64, 8, 2, 128, 128, False, FP4, 32, seed=9)
    a = r.args()
    echo.echo_qk_norm_rope(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        echo.echo_qk_norm_rope(a)
    r.qo.fill_(7.0), r.ko.fill_(7.0), r.vo.fill_(7.0)
    r.rows.copy_(dev(r.rows_np.view(np.int16)))
    g.replay()
    r.check()
