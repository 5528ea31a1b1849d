"""Pins of the gate, permute-gradient and combine-gradient oracles: hand examples and
central differences."""

import numpy as np
import pytest

import oracle as O
from oracle.combine import bf16_bits_to_f32, f32_to_bf16_bits

SOFTMAX, SIGMOID = 0, 1


def test_gate_hand_examples():
    x = np.log(np.array([[[1.0, 3.0, 4.0, 2.0]]]))
    ids, w = O.gate(x, 2, score=SOFTMAX, renorm=False)
    assert ids.tolist() == [[[2, 1]]] and np.allclose(w, [[[0.4, 0.3]]])
    ids, w = O.gate(x, 2, score=SOFTMAX, renorm=True, scale=2.0)
    assert np.allclose(w, [[[8 / 7, 6 / 7]]])
    # sigmoid(log a) = a / (1 + a): 1/2, 3/4, 4/5, 2/3; the bias lifts expert 0 to the top
    ids, w = O.gate(x, 2, bias=np.array([1.0, 0, 0, 0]), score=SIGMOID, renorm=False)
    assert ids.tolist() == [[[0, 2]]] and np.allclose(w, [[[0.5, 0.8]]])


def test_gate_masks_ties_and_absent_tokens():
    inf = np.inf
    x = np.array([[[1.0, 1.0, -inf, 1.0], [np.nan, -inf, inf, -inf], [-inf, 5.0, -inf, 4.0],
                   [0.0, -0.0, 0.0, 0.0]]])
    ids, w = O.gate(x, 3, batch_size=np.array([4]))
    assert ids[0].tolist() == [[0, 1, 3], [-1, -1, -1], [1, 3, -1], [0, 1, 2]]
    assert np.allclose(w[0, 0], 1 / 3) and (w[0, 1] == 0).all() and w[0, 2, 2] == 0
    ids, w = O.gate(x, 3, batch_size=np.array([1]))
    assert (ids[0, 1:] == -1).all() and (w[0, 1:] == 0).all()


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(score, renorm):
    """Central differences of sum(dw * w): truncation h^2 |f'''| / 6 and rounding
    2^-52 |f| / h, with |f| and its derivatives below 10 here: 1e-9 at h = 2e-5."""
    rng = np.random.default_rng(5)
    x = rng.permutation(24).reshape(1, 2, 12) / 4.0 - 3.0        # no selection changes within h
    dw = rng.standard_normal((1, 2, 3))
    ids, w = O.gate(x, 3, score=score, renorm=renorm, scale=1.7)
    got = O.gate_grad(dw, x, ids, w, score, renorm, 1.7)
    h, num = 2e-5, np.zeros_like(x)
    for i in np.ndindex(x.shape):
        f = []
        for s in (h, -h):
            y = x.copy()
            y[i] += s
            ids2, w2 = O.gate(y, 3, score=score, renorm=renorm, scale=1.7)
            assert np.array_equal(ids2, ids)
            f.append((dw * w2).sum())
        num[i] = (f[0] - f[1]) / (2 * h)
    assert np.abs(num - got).max() < 2e-8


def test_row_gradients_against_differences():
    """The combine is linear in the expert outputs and in the weights, so a difference with a
    step of 1 in 64 bits is exact up to rounding."""
    rng = np.random.default_rng(6)
    R, T, K, P, H = 2, 3, 2, 14, 8
    d = np.full(R * T * K, -1)
    d[:10] = rng.permutation(P)[:10]
    d = d.reshape(R, T, K)[::-1]
    dy = f32_to_bf16_bits(rng.standard_normal((R, T, H)).astype(np.float32))
    out = f32_to_bf16_bits(rng.standard_normal((P, H)).astype(np.float32))
    w = rng.random((R, T, K)).astype(np.float32)

    def loss(o, wt):                   # <dy, combine(o, wt)>, straight from the definition
        s = 0.0
        for r, t, k in np.ndindex(R, T, K):
            if d[r, t, k] >= 0:
                s += float(wt[r, t, k]) * (bf16_bits_to_f32(dy[r, t]).astype(np.float64)
                                           * o[d[r, t, k]]).sum()
        return s

    o64 = bf16_bits_to_f32(out).astype(np.float64)
    dout, dw, _ = O.combine_grad(dy, out, d, w)
    base = loss(o64, w.astype(np.float64))
    for i in np.ndindex(R, T, K):
        w2 = w.astype(np.float64)
        w2[i] += 1.0
        assert abs(loss(o64, w2) - base - dw[i]) < 1e-12
    for i in np.ndindex(P, H):
        o2 = o64.copy()
        o2[i] += 1.0
        want = loss(o2, w.astype(np.float64)) - base
        assert dout[i] == f32_to_bf16_bits(np.float32(want))        # rounded to bf16 once
    # the permute copies x[r][t] to its rows, so dx is the sum of the rows' gradients
    dx = O.permute_grad(out, d)
    for r, t in np.ndindex(R, T):
        rows = [j for j in d[r, t] if j >= 0]
        assert np.array_equal(dx[r, t], f32_to_bf16_bits(o64[rows].sum(0).astype(np.float32)))


@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_gradient_keeps_its_digits_near_one(renorm):
    """ds/dl = exp(-l) / (1 + exp(-l))^2, for one slot without renormalisation and, with it, of
    s0 / (s0 + s1) in s0; products and quotients of a few terms in 64 bits."""
    for top in (12.0, 30.0, 45.0):
        x = np.array([[[top, 0.5, -3.0]]])
        ids, w = O.gate(x, 2, score=SIGMOID, renorm=renorm)
        assert ids.tolist() == [[[0, 1]]]
        d = O.gate_grad(np.array([[[1.0, 0.0]]]), x, ids, w, SIGMOID, renorm)[0, 0]
        e0, e1 = np.exp(-top), np.exp(-0.5)
        ds, s0, s1 = e0 / (1 + e0) ** 2, 1 / (1 + e0), 1 / (1 + e1)
        want = ds * s1 / (s0 + s1) ** 2 if renorm else ds
        assert abs(d[0] / want - 1) < 1e-13 and d[2] == 0


def test_sigmoid_without_a_bias_orders_by_the_logits():
    x = np.array([[[40.0, 800.0, -900.0, -800.0, 41.0]]])        # scores 1, 1, 0, 0, 1 in 64 bits
    assert O.gate(x, 5, score=SIGMOID)[0].tolist() == [[[1, 4, 0, 3, 2]]]
    assert O.gate(x, 3, bias=np.zeros(5), score=SIGMOID)[0].tolist() == [[[0, 1, 4]]]
