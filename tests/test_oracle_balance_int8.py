"""Pins of the oracle's balance loss, rows in 8 bits and products (CPU)."""

import numpy as np
import pytest

import oracle as O


def test_balance_by_hand():
    """Two tokens, two experts, K = 1: p = (3/4, 1/4) and (1/2, 1/2), both routed to expert 0:
    counts (2, 0), prob (5/8, 3/8), loss = 2 / (1 * 2) * 2 * 5/8 = 1.25."""
    logits = np.log(np.array([[[3.0, 1.0], [1.0, 1.0]]]))
    loss, counts, prob, tokens = O.balance_loss(logits, np.array([[[0], [0]]]))
    assert counts.tolist() == [[2, 0]] and tokens.tolist() == [2]
    assert np.allclose(prob, [[5 / 8, 3 / 8]]) and np.allclose(loss, [1.25])
    # a third token is absent: nothing changes
    more = np.concatenate([logits, [[[5.0, -5.0]]]], axis=1)
    loss2, _, _, tokens2 = O.balance_loss(more, np.array([[[0], [0], [-1]]]))
    assert tokens2.tolist() == [2] and np.allclose(loss2, loss)


@pytest.mark.parametrize("score", [0, 1])
def test_an_even_load_has_loss_one(score):
    ids = np.arange(8).reshape(1, 4, 2)
    loss, _, prob, _ = O.balance_loss(np.zeros((1, 4, 8)), ids, score=score)
    assert np.allclose(prob, 1 / 8) and np.allclose(loss, 1.0)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("offset", [None, [1, 1, 5, 9]])
def test_gradient_against_differences(score, offset):
    rng = np.random.default_rng(score)
    R, T, E, K, G = 1, 12, 5, 2, 3
    x = rng.normal(size=(R, T, E))
    x[0, 3, 2] = -np.inf
    ids = np.argsort(-np.where(np.isfinite(x), x, -9), axis=-1)[..., :K]
    ids[0, 2] = -1
    ids[0, 7, 1] = -1
    dloss = rng.normal(size=G)
    _, counts, _, tokens = O.balance_loss(x, ids, G, offset, score)
    got = O.balance_loss_grad(dloss, x, ids, counts, tokens, G, offset, score)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(x[0, t, e]):
                assert got[0, t, e] == 0
                continue
            up, dn = x.copy(), x.copy()
            up[0, t, e] += h
            dn[0, t, e] -= h
            d = (O.balance_loss(up, ids, G, offset, score)[0]
                 - O.balance_loss(dn, ids, G, offset, score)[0]) @ dloss / (2 * h)
            assert abs(d - got[0, t, e]) < 1e-8


def test_rows_in_8_bits_by_hand():
    x = np.array([[127.0, 0.5, 1.5, -2.5, -0.4], [0, 0, 0, 0, 0],
                  [np.nan, np.inf, -np.inf, 254.0, -3.0]])
    q, s = O.quant_rows(x)
    assert s.dtype == np.float32 and s.tolist() == [1.0, 2.0 ** -126, 2.0]
    assert q.tolist() == [[127, 0, 2, -2, 0], [0] * 5, [0, 127, -127, 127, -2]]


def test_product_by_hand():
    """One rank, one main and one slot: row 0 by the main, row 1 by the slot's weights."""
    q = np.array([[1, 2], [3, -4]], dtype=np.int8)
    w = np.array([[[1, 1], [2, -1]]], dtype=np.int8)
    slot = np.array([[[[5, 0], [0, 5]]]], dtype=np.int8)
    parts = O.expert_product(q, np.array([1.0, 0.5]), [0, 1, 2], 1, 1, 1, w, np.array([[1.0, 2.0]]),
                             slot, np.array([[[1.0, 1.0]]]))
    assert [y.tolist() for _, y, _ in parts] == [[[3.0, 0.0]], [[7.5, -10.0]]]
    (_, y, gate), _ = O.expert_product(q, np.array([1.0, 0.5]), [0, 1, 2], 1, 1, 1, w,
                                       np.array([[1.0, 2.0]]), slot, np.array([[[1.0, 1.0]]]),
                                       swiglu=True)
    assert gate.tolist() == [[3.0]] and y.tolist() == [[0.0]]
