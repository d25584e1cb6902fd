"""The expert-by-expert form of the routed oracle against its pair-by-pair form, and its gates of large logits."""
import numpy as np
import pytest

from oracle import few


@pytest.mark.parametrize("own_terms", [False, True])
def test_by_expert_is_pair_by_pair(own_terms):
    rng = np.random.default_rng(5)
    T, d, F, E, k = 9, 24, 16, 4, 5
    x, w13, w2 = rng.standard_normal((T, d)), rng.standard_normal((E, 2 * F, d)), rng.standard_normal((E, d, F))
    idx = rng.integers(-1, E + 1, (T, k))        # some outside [0, E), some twice in a row
    idx[3] = -1
    gates = rng.random((T, k))
    terms = (np.abs(w13) * 3, np.abs(w2) * 5) if own_terms else ()
    ref, bound = few.moe_swiglu_by_expert(x, idx, gates, w13, w2, *terms)
    np.testing.assert_allclose(ref, few.moe_swiglu(x, idx, gates, w13, w2), rtol=1e-11, atol=1e-11)
    np.testing.assert_allclose(bound, few.moe_swiglu_bound(x, idx, gates, w13, w2, *terms), rtol=1e-9, atol=1e-18)
    assert not ref[3].any() and not bound[3].any()


def test_sigmoid_gates_keep_their_proportions():
    l = np.array([[-999.0, -1000.0, -1000.0 - np.log(2.0), -3000.0]])
    idx, gates = few.moe_choose(l, 3, "sigmoid", True, 2.0)
    e = np.exp(-1.0)
    np.testing.assert_allclose(gates[0], 2.0 * np.array([1.0, e, e / 2]) / (1 + 1.5 * e), rtol=1e-12)
    _, gates = few.moe_choose(np.array([[3.0, -2.0]]), 2, "sigmoid", False)
    np.testing.assert_allclose(gates[0], [1 / (1 + np.exp(-3.0)), 1 / (1 + np.exp(2.0))], rtol=1e-14)
