"""CPU checks of the bounds that the softmax attention's oracle derives."""
import numpy as np
import pytest

from oracle import softmax_attention as att


@pytest.mark.parametrize("hq,hk,nq,nk,terms", [(6, 2, 5, 11, 15), (6, 2, 5, 40, 40), (8, 1, 9, 3, 72),
                                               (2, 2, 7, 4, 7)])
def test_terms_of_the_gradients_sums(monkeypatch, hq, hk, nq, nk, terms):
    """dK and dV sum over the queries of every head of a group, dQ over the keys: the longer of
    the two counts."""
    rng = np.random.default_rng(1)
    Q, dO = (rng.standard_normal((1, hq, nq, 8)) for _ in range(2))
    K, V = (rng.standard_normal((1, hk, nk, 8)) for _ in range(2))
    seen = set()
    monkeypatch.setattr(att, "_sums", lambda n: seen.add(n) or 0.0)
    att.backward(Q, K, V, dO)
    assert seen == {terms}
