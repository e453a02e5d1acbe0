"""The bound on bf16 attention that the GPU tests use tells two-term softmax weights from one
bf16 term, on the values those tests use.  No GPU needed."""
import numpy as np
import pytest

import block_ref as ref


@pytest.mark.parametrize("n", [2, 6, 40, 130])
@pytest.mark.parametrize("D", [64, 128])
def test_the_bound_holds_for_two_terms_and_not_for_one(n, D):
    g = np.random.default_rng(n + D)
    q = ref.bf16_round(0.02 * g.standard_normal((8, D)))
    k, v = ref.bf16_round(g.standard_normal((n, D))), ref.opposite_values(g, n, D)
    want = ref.attention(q, [(k, v)] * 8, D ** -0.5)
    far = ref.two_term_bounds(D, np.full(8, n), *want)
    x = q @ k.T * D ** -0.5
    p = np.exp(x - x.max(1, keepdims=True))
    one = ref.bf16_round(p)
    two = one + ref.bf16_round(p - one)
    err = lambda w: np.abs(ref.bf16_round(w @ v / p.sum(1, keepdims=True)) - want[0])
    assert (err(two) <= far).all()
    assert (err(one) > far).mean() > 0.2
