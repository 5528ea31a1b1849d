"""Oracle: the router's balance loss and its gradient, in 64 bits.

UltraEP article, section "在 Gate 之后获取当前层真实负载": the path balances the load that the Gate
has produced; the auxiliary loss that trains a Gate towards an even load is the article's point
of comparison and is not written out there.  The reading here is the standard one: for the
tokens of a sequence, n of them present (some id >= 0),

  * p = softmax of the logits, or sigmoid scores divided by their sum over the experts;
  * counts_e = ids of expert e, prob_e = mean of p_e over the present tokens;
  * loss = E / (K n) * sum_e counts_e prob_e, 0 for a sequence without tokens;
  * gradient: the counts held fixed, absent tokens 0.

Only finite logits have a score.  Pins (tests/test_oracle_balance_int8.py): a hand example, the
value 1 of an even load, the gradient against central differences.  Parity with a source's
numbers: unpinned (the pages give none).
"""

import numpy as np

from .gate import SIGMOID, _scores, _sigmoid


def spans(n_tok, n_seq=1, seq_offset=None):
    """[first, end) of every sequence."""
    if seq_offset is None:
        return [(n_tok // n_seq * g, n_tok // n_seq * (g + 1)) for g in range(n_seq)]
    return [(int(a), int(b)) for a, b in zip(seq_offset[:-1], seq_offset[1:])]


def balance_shares(logits, score):
    """p of every token (0 where no logit is finite) and its scores, [n][E]."""
    s, _ = _scores(np.asarray(logits), score)
    s = s.reshape(-1, s.shape[-1])
    z = s.sum(-1, keepdims=True)
    return s / np.where(z > 0, z, 1.0), s


def balance_loss(logits, topk_ids, n_seq=1, seq_offset=None, score=0):
    """loss [n_seq], counts [n_seq][E] int64, prob [n_seq][E], tokens [n_seq] int64."""
    E, K = np.asarray(logits).shape[-1], np.asarray(topk_ids).shape[-1]
    p, _ = balance_shares(logits, score)
    ids = np.asarray(topk_ids).reshape(-1, K)
    live = (ids >= 0).any(1)
    loss, counts, prob, tokens = [], [], [], []
    for a, b in spans(len(ids), n_seq, seq_offset):
        part = ids[a:b][ids[a:b] >= 0]
        counts.append(np.bincount(part, minlength=E))
        n = int(live[a:b].sum())
        tokens.append(n)
        prob.append(p[a:b][live[a:b]].sum(0) / max(n, 1))
        loss.append(E / (K * max(n, 1)) * float((counts[-1] * prob[-1]).sum()))
    return np.array(loss), np.array(counts), np.array(prob), np.array(tokens)


def balance_loss_grad(dloss, logits, topk_ids, counts, tokens, n_seq=1, seq_offset=None, score=0):
    """dlogits [R][T][E]; tokens outside of every sequence get 0."""
    shape = np.asarray(logits).shape
    E, K = shape[-1], np.asarray(topk_ids).shape[-1]
    p, s = balance_shares(logits, score)
    x = np.asarray(logits, dtype=np.float64).reshape(-1, E)
    live = (np.asarray(topk_ids).reshape(-1, K) >= 0).any(1)
    out = np.zeros_like(p)
    for g, (a, b) in enumerate(spans(len(p), n_seq, seq_offset)):
        n = float(tokens[g])
        if n <= 0:
            continue
        c = np.asarray(counts[g], dtype=np.float64)
        # about the count of the likeliest expert, next to which differences keep their digits
        c0 = c[p[a:b].argmax(-1)][:, None]
        d = p[a:b] * ((c - c0) - (p[a:b] * (c - c0)).sum(-1, keepdims=True))
        if score == SIGMOID:
            with np.errstate(over="ignore"):
                d = d * np.where(np.isfinite(x[a:b]), _sigmoid(-np.where(np.isfinite(x[a:b]), x[a:b], 0)), 0)
        out[a:b] = float(dloss[g]) * E / (K * n * n) * d * live[a:b, None]
    return out.reshape(shape)
