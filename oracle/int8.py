"""Oracle: rows in 8 bits and the experts' products on them, in 64 bits.

The pages leave the experts' products to the model; the reading here is the standard symmetric
one with a scale for each row and each output channel:

  * scale = max(fp32(largest finite |x| / 127), 2^-126), q = x / scale to the nearest integer
    (ties to even), NaN 0 and an infinity +-127;
  * y[p][n] = (sum_d q[p][d] w[n][d]) * w_scale[n] * q_scale[p] with the weights of the row's
    instance; SwiGLU: silu(first half) * second half.

Instances as in UltraEP's shared redundant slots ("共享冗余 slot 管理动态专家副本"): instance
r * (E/R + S) + j is main r * E/R + j for j < E/R, else slot (r, j - E/R).  Pins
(tests/test_oracle_balance_int8.py): hand examples.  Parity with a source's numbers: unpinned.
"""

import numpy as np


def quant_rows(x):
    """q int8 and scale float32 of the rows of x (any float type that holds bf16 values)."""
    x = np.asarray(x, dtype=np.float64)
    able = np.isfinite(x)
    top = np.where(able, np.abs(x), 0.0).max(-1)
    scale = np.maximum((top / 127.0).astype(np.float32), np.float32(2.0 ** -126))
    with np.errstate(invalid="ignore"):
        q = np.rint(np.where(able, x, 0.0) / scale.astype(np.float64)[..., None])
        q = np.where(np.isinf(x), np.copysign(127.0, x), q)
    return q.astype(np.int8), scale


def expert_product(q, q_scale, offset, R, E, S, main_w, main_scale, slot_w=None, slot_scale=None,
                   swiglu=False):
    """(rows, y) of every instance with rows: y float64 [n][N or N/2], gate float64 or None."""
    per = E // R + S
    out = []
    for i in range(R * per):
        a, b = int(offset[i]), int(offset[i + 1])
        if a == b:
            continue
        r, j = divmod(i, per)
        w, s = (main_w[r * (E // R) + j], main_scale[r * (E // R) + j]) if j < E // R else \
            (slot_w[r][j - E // R], slot_scale[r][j - E // R])
        z = q[a:b].astype(np.float64) @ np.asarray(w, dtype=np.float64).T     # exact: below 2^53
        y = z * np.asarray(s, dtype=np.float64) * np.asarray(q_scale[a:b], dtype=np.float64)[:, None]
        gate = None
        if swiglu:
            gate, up = np.split(y, 2, axis=-1)
            with np.errstate(over="ignore"):
                y = gate / (1.0 + np.exp(-gate)) * up
        out.append((slice(a, b), y, gate))
    return out
