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


@pytest.mark.parametrize("kw", [{}, dict(causal=True, window=4, q_lengths=[5], k_lengths=[8])])
def test_gradients_with_the_forwards_result(kw):
    """With the exact O they are the same; a rounded O changes dQ and dK as
    scale sum_j p_ij (delta_i - delta'_i) K_j says, within the part of the bounds for it."""
    rng = np.random.default_rng(2)
    Q, dO = (rng.standard_normal((1, 4, 6, 8)) for _ in range(2))
    K, V = (rng.standard_normal((1, 2, 9, 8)) for _ in range(2))
    O = att.forward(Q, K, V, **kw)[0]
    plain, bounds, rows = att.backward(Q, K, V, dO, **kw)
    same, tighter, none = att.backward(Q, K, V, dO, O=O, **kw)
    for a, b in zip(plain, same):
        assert np.allclose(a, b, rtol=1e-12, atol=1e-13)
    assert all((x == 0).all() for x in none) and all((x <= y).all() for x, y in zip(tighter, bounds))
    off = O * (1 + att.U * rng.uniform(-1, 1, O.shape))
    moved = att.backward(Q, K, V, dO, O=off, **kw)[0]
    assert not np.allclose(moved[0], plain[0], rtol=1e-9)
    for a, b, r in zip(moved, plain, rows):
        assert (np.abs(a - b) <= r * (1 + 1e-9) + 1e-15).all()
