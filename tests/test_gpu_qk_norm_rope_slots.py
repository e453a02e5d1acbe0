"""echo_qk_norm_rope: a slot that two tokens of a call share."""
import numpy as np
import pytest
import torch

import sparse_attention_kv_fp8_gb300 as echo
from helpers import dev
from test_gpu_qk_norm_rope import BF16, FP4, Rope

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("T", [2, 600])
def test_a_shared_slot_holds_bytes_of_its_tokens_and_touches_no_other(fmt, T):
    r = Rope(T, 4, 3, 128, 64, False, fmt, 16, seed=4)
    half = T // 2
    r.slot_np[half:] = r.slot_np[:half]
    rows = []
    for part in (slice(0, T), slice(0, half), slice(half, T)):    # both, and each alone
        slot = np.full(T, -1, np.int32)
        slot[part] = r.slot_np[part]
        r.rows.copy_(dev(r.rows_np.view(np.int16)))
        echo.echo_qk_norm_rope(r.args(slot_map=dev(slot)))
        torch.cuda.synchronize()
        rows.append(r.rows.cpu().numpy().view(np.uint8))
    both, first, second = rows
    assert ((both == first) | (both == second)).all() and int(r.status) == 0
