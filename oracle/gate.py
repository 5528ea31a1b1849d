"""Oracle: the router gate and its gradient, in 64 bits.

UltraEP article, section "在 Gate 之后获取当前层真实负载": the balancing path starts from the
routing that the layer's Gate has produced.  The pages do not write the Gate out; the
reading here is the standard one of the layers they measure (softmax over all experts, or
sigmoid with a selection bias, top-k, optionally renormalised weights):

  * scores s_e = exp(l_e) / sum_j exp(l_j), or s_e = 1 / (1 + exp(-l_e));
  * selection by l_e, or by s_e + bias_e where a bias is given, descending, ties to the lowest
    id (a sigmoid without a bias orders like its logits, also where its scores round alike);
  * w_k = scale * s_k, or scale * s_k / (sum over the selected s), 0 if that sum is 0;
  * only finite logits (and finite s_e + bias_e) are eligible; slots past the eligible
    experts, and absent tokens, hold id -1 and weight 0.

Pins (tests/test_oracle_gate_grads.py): a hand example of each score; the gradient
against central differences of the weights.  Parity with a source's numbers: unpinned
(the pages give none).
"""

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _scores(logits, score):
    x = np.asarray(logits, dtype=np.float64)
    able = np.isfinite(x)
    safe = np.where(able, x, 0.0)
    if score == SIGMOID:
        return np.where(able, _sigmoid(safe), 0.0), able
    top = np.max(np.where(able, x, -np.inf), axis=-1, keepdims=True)
    e = np.where(able, np.exp(safe - np.where(np.isfinite(top), top, 0.0)), 0.0)
    z = e.sum(-1, keepdims=True)
    return e / np.where(z > 0, z, 1.0), able


def gate_keys(logits, bias=None, score=SOFTMAX):
    """What the selection orders by; -inf where an expert is not eligible."""
    s, able = _scores(logits, score)
    key = np.asarray(logits, dtype=np.float64) if score == SOFTMAX or bias is None else \
        s + np.asarray(bias, dtype=np.float64)
    return np.where(able & np.isfinite(key), key, -np.inf)


def gate(logits, K, bias=None, batch_size=None, score=SOFTMAX, renorm=True, scale=1.0):
    """topk_ids int32 [R][T][K] and weights float64 [R][T][K] for logits [R][T][E]."""
    R, T, _ = np.asarray(logits).shape
    key = gate_keys(logits, bias, score)
    order = np.argsort(-key, axis=-1, kind="stable")[..., :K]
    live = np.take_along_axis(key, order, -1) > -np.inf
    if batch_size is not None:
        live &= (np.arange(T)[None, :] < np.asarray(batch_size)[:, None])[..., None]
    s, _ = _scores(logits, score)
    w = np.where(live, np.take_along_axis(s, order, -1), 0.0)
    if renorm:
        z = w.sum(-1, keepdims=True)
        w = w / np.where(z > 0, z, 1.0)
    return np.where(live, order, -1).astype(np.int32), w * scale


def gate_grad(dgate_w, logits, topk_ids, gate_w, score=SOFTMAX, renorm=True, scale=1.0):
    """dlogits float64 [R][T][E]: the chain rule through gate's weights with the selection
    held fixed (gate_w as gate returned it)."""
    s, able = _scores(logits, score)
    ids = np.asarray(topk_ids)
    on = ids >= 0
    at = np.where(on, ids, 0)
    picked = np.take_along_axis(np.where(able, np.asarray(logits, dtype=np.float64), 0.0), at, -1)
    rest = _sigmoid(-picked)                # 1 - s, which as a difference loses digits near 1
    g = np.where(on, np.asarray(dgate_w, dtype=np.float64) * scale, 0.0)
    u = np.where(on, np.asarray(gate_w, dtype=np.float64) / scale, 0.0)
    dot = (u * g).sum(-1, keepdims=True)
    if renorm:
        d = u * (g - dot)
        if score == SIGMOID:
            d = d * rest
    else:
        d = u * rest * g if score == SIGMOID else g
    out = np.zeros(s.shape)
    for k in range(ids.shape[-1]):
        r, t = np.nonzero(on[..., k])
        out[r, t, ids[r, t, k]] += d[r, t, k]
    if score == SOFTMAX and not renorm:
        out = s * (out - dot) * on.any(-1, keepdims=True)
    return out
