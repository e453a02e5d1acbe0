"""echo_block_tables on the GPU against its definition, one block at a time on the CPU:
every output equal, untouched entries untouched."""
import numpy as np
import pytest
import torch

import block_ref as ref
import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, old, new, bs, seed=0, n_free=None, max_new=None, max_blocks=None, n_blocks=None, shift=0):
        g = np.random.default_rng(seed)
        self.old, self.new, self.bs = np.array(old, np.int32), np.array(new, np.int32), bs
        B, nb = len(old), -(-self.old // bs)
        mb = max_blocks or max(1, int((-(-np.maximum(self.old, self.new) // bs)).max(initial=1)))
        used = int(nb.sum())
        need = int(np.maximum(-(-self.new // bs) - nb, 0).sum())
        n_free = need + 3 if n_free is None else n_free
        self.n_blocks = n_blocks or used + n_free
        ids = g.permutation(self.n_blocks).astype(np.int32)
        self.table = np.full((B, mb), -7, np.int32)
        self.table[np.arange(mb)[None] < nb[:, None]] = ids[:used]
        self.free = np.full(self.n_blocks, -9, np.int32)
        self.free[:n_free] = ids[used:used + n_free]
        self.count = n_free
        self.max_new = int(np.maximum(self.new - self.old, 0).sum()) + 5 if max_new is None else max_new
        self.t = dict(old=dev(self.old), new=dev(self.new), table=dev(self.table), free=dev(self.free),
                      count=dev(np.array([n_free], np.int32)))
        i32 = lambda n: torch.full((n,), -99, dtype=torch.int32, device="cuda")
        self.slot = i32(self.max_new + shift)[shift:]
        self.out = dict(count=i32(1), pos=i32(self.max_new), cu=i32(B + 1), len=i32(B), status=i32(1).zero_())
        self.args = echo.make_block_tables_args(self.t["old"], self.t["new"], bs, self.t["table"], self.t["free"],
                                                self.t["count"], self.out["count"], self.slot, self.out["pos"],
                                                self.out["cu"], self.out["len"], self.out["status"])

    def check(self, status=0):
        want = ref.block_tables(self.old, self.new, self.bs, self.table, self.free, self.count, self.max_new)
        torch.cuda.synchronize()
        got = (self.t["table"], self.t["free"], self.out["count"], self.slot, self.out["pos"], self.out["cu"],
               self.out["len"])
        for name, a, b in zip(("table", "free", "count", "slot", "pos", "cu", "len"), got, want):
            assert np.array_equal(a.cpu().numpy(), np.atleast_1d(b)), name
        st = status | (echo.DEV_POOL_EXHAUSTED if want[-1] else 0)
        assert int(self.out["status"]) == st


def lengths(B, L, new, seed):
    g = np.random.default_rng(seed)
    old = g.integers(0, L + 1, B)
    return old, np.maximum(0, old + g.integers(-new, new + 1, B))


@pytest.mark.parametrize("old,new,bs", [
    ([0], [1], 16), ([0], [0], 16), ([63], [64], 64), ([64], [65], 64), ([65], [64], 64), ([64], [63], 64),
    ([1], [0], 64), ([5, 0, 9], [0, 0, 0], 4), ([0, 0, 0], [5, 0, 9], 4), ([7, 7], [7, 7], 4),
    ([100, 3, 0, 17, 64], [90, 40, 128, 0, 65], 16), ([0] * 40, [1] * 40, 1),
])
def test_small_steps(old, new, bs):
    s = Step(old, new, bs)
    echo.echo_block_tables(s.args)
    s.check()


@pytest.mark.parametrize("B,L,new,bs", [(1, 40000, 20000, 64), (37, 900, 1, 64), (64, 32768, 2, 64), (511, 50, 60, 16),
                                        (513, 300, 300, 7), (2000, 100, 5, 16), (16384, 30, 9, 16),
                                        (100, 10000, 9000, 64), (90, 9000, 9000, 3), (16000, 80, 60, 2)])
@pytest.mark.parametrize("seed", [1, 2])
def test_random_steps(B, L, new, bs, seed):
    s = Step(*lengths(B, L, new, seed), bs, seed)
    echo.echo_block_tables(s.args)
    s.check()


@pytest.mark.parametrize("B,L,bs", [(300, 3000, 4), (40, 30000, 16), (700, 900, 1)])
def test_finished_requests_return_all_their_blocks(B, L, bs):
    """Nine in ten end, the others go on by a token: far more blocks move than tokens come."""
    old = np.random.default_rng(B).integers(0, L + 1, B)
    s = Step(old, np.where(np.arange(B) % 10 == 3, old + 1, 0), bs, 4)
    for _ in range(2):
        echo.echo_block_tables(s.args)
    s.check()


@pytest.mark.parametrize("short", [1, 3, 1000])
def test_growth_that_does_not_fit_is_left_out_in_order(short):
    old, new = lengths(200, 400, 200, 5)
    need = np.maximum(-(-new // 16) - -(-old // 16), 0).sum()
    freed = np.maximum(-(-old // 16) - -(-new // 16), 0).sum()
    s = Step(old, new, 16, 5, n_free=max(0, int(need - freed) - short))
    echo.echo_block_tables(s.args)
    s.check()


def test_freed_blocks_serve_the_same_step_and_a_step_back_restores_nothing_else():
    s = Step([64, 0, 48], [0, 80, 48], 16, 3, n_free=2)      # 4 freed + 2: the 5 needed fit
    echo.echo_block_tables(s.args)
    s.check()


def test_a_repeated_call_gives_the_same_outputs():
    s = Step(*lengths(100, 500, 300, 9), 32, 9)
    for _ in range(3):
        echo.echo_block_tables(s.args)
    s.check()


@pytest.mark.parametrize("shift", [1, 3])
def test_unaligned_lists_and_too_few_entries(shift):
    s = Step([0, 10], [50, 90], 16, 4, shift=shift)
    echo.echo_block_tables(s.args)
    s.check()
    s = Step([0, 10], [50, 90], 16, 4, max_new=77, shift=shift)   # 130 new tokens, 77 entries
    echo.echo_block_tables(s.args)
    s.check(echo.DEV_BAD_INDEX)
    s = Step([3], [3], 16, 4, max_new=0)
    echo.echo_block_tables(s.args)
    s.check()
    s = Step(*lengths(70, 9000, 9000, 3), 16, 3, shift=shift)
    echo.echo_block_tables(s.args)
    s.check()
    s = Step([], [], 16, 3, n_free=2, n_blocks=2)
    echo.echo_block_tables(s.args)
    s.check()


def test_bad_lengths_and_counts_are_clamped_and_flagged():
    """Lengths past the table or negative act as the nearest legal ones; a stack height
    outside the stack likewise."""
    s = Step([10, 20, 30], [40, 0, 48], 16, 6, max_blocks=3, n_free=4)
    s.t["new"].copy_(dev(np.array([40, -5, 4000], np.int32)))
    echo.echo_block_tables(s.args)
    s.check(echo.DEV_BAD_INDEX)
    s = Step([10], [40], 16, 6, n_free=4, n_blocks=5)
    s.t["count"].fill_(-3)
    s.count = 0
    echo.echo_block_tables(s.args)
    s.check(echo.DEV_BAD_INDEX)


def test_ids_outside_the_pool_are_not_handed_out():
    s = Step([0], [40], 16, 7, n_free=4)
    s.t["free"].fill_(1 << 30)
    echo.echo_block_tables(s.args)
    torch.cuda.synchronize()
    assert int(s.out["status"]) == echo.DEV_BAD_INDEX and bool((s.slot == -1).all()) and bool((s.out["pos"] == -1).all())


def test_captured_steps_on_another_stream():
    """Two steps in turn (counters swapped), captured once on a side stream and replayed."""
    a = Step([60, 5], [64, 30], 16, 8, n_free=12)
    i32 = lambda n: torch.full((n,), -99, dtype=torch.int32, device="cuda")
    new2, slot2, count2 = dev(np.array([70, 31], np.int32)), i32(10), i32(1)
    a.t["table"] = dev(np.pad(a.table, ((0, 0), (0, 2)), constant_values=-7))
    args1 = echo.make_block_tables_args(a.t["old"], a.t["new"], 16, a.t["table"], a.t["free"], a.t["count"],
                                        a.out["count"], a.slot)
    args2 = echo.make_block_tables_args(a.t["new"], new2, 16, a.t["table"], a.t["free"], a.out["count"], count2, slot2)
    echo.echo_block_tables(args1)
    torch.cuda.synchronize()
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        echo.echo_block_tables(args1)
        echo.echo_block_tables(args2)
    g.replay()
    torch.cuda.synchronize()
    table = np.pad(a.table, ((0, 0), (0, 2)), constant_values=-7)
    t1, f1, n1, s1, *_ = ref.block_tables(a.old, a.new, 16, table, a.free, a.count, a.max_new)
    t2, f2, n2, s2, *_ = ref.block_tables(a.new, [70, 31], 16, t1, f1, n1, 10)
    assert np.array_equal(a.t["table"].cpu().numpy(), t2) and int(count2) == n2
    assert np.array_equal(a.slot.cpu().numpy(), s1) and np.array_equal(slot2.cpu().numpy(), s2)
