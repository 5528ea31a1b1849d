"""Oracle: gradients of the permute and of the combine.

UltraEP article, section "复用前向方案，完成权重恢复与梯度归约": backward reuses the forward
plan.  With y[g] = sum_k w[g][k] out[row(g, k)] (oracle/combine.py) and out[row(g, k)] =
x[g] (oracle/permute.py), the chain rule gives

    dout[row(g, k)] = w[g][k] dy[g]          dw[g][k] = <dy[g], out[row(g, k)]>
    dx[g] = sum_k dout[row(g, k)]

over the slots that have a row.  dx has the combine's arithmetic with every weight 1 and
dout is one fp32 product rounded to bf16, so both can be matched bit for bit; dw is a 64-bit
sum here.

Pins (tests/test_oracle_gate_grads.py): all three against differences of the forward
functions, which are linear in each argument.
"""

import numpy as np

from .combine import bf16_bits_to_f32, combine, f32_to_bf16_bits


def permute_grad(dout_bits, dest_row, r_begin=0, r_end=None):
    """dx bf16 bits [R][T][H] (0 outside the rank range)."""
    return combine(dout_bits, dest_row, np.ones(dest_row.shape, dtype=np.float32), r_begin, r_end)


def combine_grad(dy_bits, out_bits, dest_row, gate_w):
    """dout bf16 bits [P][H] (rows without a slot stay 0), dgate_w float64 [R][T][K], and the
    sum of the dot products' magnitudes [R][T][K] (for error bounds)."""
    R, T, K = dest_row.shape
    P, H = out_bits.shape
    dy = bf16_bits_to_f32(dy_bits.reshape(R * T, H))
    d, w = dest_row.reshape(R * T, K), gate_w.reshape(R * T, K).astype(np.float32)
    dout = np.zeros((P, H), dtype=np.uint16)
    dw, mag = np.zeros((R * T, K)), np.zeros((R * T, K))
    for k in range(K):
        g = np.nonzero(d[:, k] >= 0)[0]
        rows = d[g, k]
        with np.errstate(over="ignore", invalid="ignore"):
            dout[rows] = f32_to_bf16_bits(w[g, k][:, None] * dy[g])
            term = dy[g].astype(np.float64) * bf16_bits_to_f32(out_bits[rows]).astype(np.float64)
            dw[g, k], mag[g, k] = term.sum(-1), np.abs(term).sum(-1)
    return dout, dw.reshape(R, T, K), mag.reshape(R, T, K)
