"""Oracle: the AdamW step, states in fp32 or in 8 bits with stochastic rounding.

UltraEP article, section "共享冗余 slot 管理动态专家副本": redundant slots carry no optimizer
state; the mains are stepped after the gradient reduction.  The pages name no optimizer;
the reading is AdamW (decoupled weight decay, bias-corrected moments).  m and v are fixed
to the bit (fp32, each product and sum rounded on its own); the parameter's update is a
64-bit value here.

8-bit states: an fp32 number's level is its upper 11 bits below the sign (8 of exponent, 3
of mantissa) after a random number of 2^-16 steps was added; a block of 256 elements stores
its largest level and each element's distance below it.

Pins (tests/test_oracle_adamw.py): torch.optim.AdamW in float64; the rounding against its
definition by real numbers (the level is floor(8 log-linear position + dither)), its mean
over the dither, and the uniformity of the random halves.
"""

import numpy as np

BLOCK = 256
M32 = np.uint64(0xFFFFFFFF)


def _mix(x):
    x = np.asarray(x, dtype=np.uint64) & M32
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x9E3779B9)) & M32
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xBB67AE85)) & M32
    return x ^ (x >> np.uint64(16))


def _next(x):
    x = x ^ ((x << np.uint64(13)) & M32)
    x = x ^ (x >> np.uint64(17))
    return x ^ ((x << np.uint64(5)) & M32)


def dithers(seed, step, index, n):
    """16-bit random numbers of a tensor's n elements: for the parameter, for m, for v."""
    key = _mix(_mix(np.uint64((step * 0x9E3779B9 + seed) & 0xFFFFFFFF)) ^ np.uint64(index + 1))
    i = np.arange((n + 3) // 4, dtype=np.uint64)
    w = [_mix(((i * np.uint64(0x9E3779B9)) & M32) ^ key)]
    for _ in range(5):
        w.append(_next(w[-1]))
    low, high = np.uint64(0xFFFF), np.uint64(16)
    p = np.stack([w[0] & low, w[0] >> high, w[1] & low, w[1] >> high], 1).reshape(-1)[:n]
    s = np.stack(w[2:], 1).reshape(-1)[:n]
    return p.astype(np.uint32), (s & low).astype(np.uint32), (s >> high).astype(np.uint32)


def levels(x, dither):
    bits = np.abs(np.asarray(x, dtype=np.float32)).view(np.uint32)
    lv = np.minimum((bits + (dither.astype(np.uint32) << np.uint32(4))) >> np.uint32(20), 0x7F7)
    return np.where(bits > 0, lv, 0).astype(np.int64)


def _tops(lv):
    pad = np.zeros(-(-len(lv) // BLOCK) * BLOCK, dtype=np.int64)
    pad[:len(lv)] = lv
    return pad.reshape(-1, BLOCK).max(1)


def encode(m, v, dm, dv):
    """uint8 codes of m and v and int32 tops for fp32 arrays and their dithers."""
    lm, lv = levels(m, dm), levels(v, dv)
    tm, tv = _tops(lm), _tops(lv)
    n = len(lm)
    at = np.arange(n) // BLOCK
    cm = np.maximum(lm - tm[at] + 127, 0)
    cm = np.where((m != 0) & (cm > 0), cm | np.where(m < 0, 128, 0), 0)
    cv = np.where(v > 0, np.maximum(lv - tv[at] + 255, 1), 0)
    return cm.astype(np.uint8), cv.astype(np.uint8), (tm | (tv << 16)).astype(np.int32)


def _value(level):
    return (np.maximum(level, 0).astype(np.uint32) << np.uint32(20)).view(np.float32)


def decode(m_codes, v_codes, tops):
    """fp32 values of 8-bit states."""
    at = np.arange(len(m_codes)) // BLOCK
    tm, tv = (tops.astype(np.int64) & 0xFFFF)[at], (tops.astype(np.int64) >> 16)[at]
    size = (m_codes & 127).astype(np.int64)
    m = np.where(size > 0, _value(size - 127 + tm), np.float32(0))
    v = np.where(v_codes > 0, _value(v_codes.astype(np.int64) - 255 + tv), np.float32(0))
    return np.where(m_codes & 128, -m, m).astype(np.float32), v.astype(np.float32)


def moments(grad, m, v, factor, beta1=0.9, beta2=0.999):
    """New m and v in fp32, every product and sum rounded on its own (bit for bit), and which
    elements' gradients were not finite (taken as 0)."""
    f = np.float32
    with np.errstate(over="ignore", invalid="ignore"):
        g = grad.astype(f) * f(factor)
        bad = ~np.isfinite(g)
        g = np.where(bad, f(0), g).astype(f)
        m = m.astype(f) * f(beta1) + g * f(1.0 - beta1)
        v = v.astype(f) * f(beta2) + (g * g) * f(1.0 - beta2)
    return m, v, bad


def update(p, m, v, step, lr, weight_decay=0.0, beta1=0.9, beta2=0.999, eps=1e-8):
    """The new parameter from the new m and v, float64, and the size of the change."""
    p, m, v = (np.asarray(a, dtype=np.float64) for a in (p, m, v))
    hat = (m / (1.0 - beta1 ** step)) / (np.sqrt(v / (1.0 - beta2 ** step)) + eps)
    return p * (1.0 - lr * weight_decay) - lr * hat, np.abs(lr * hat)


def cut_bf16(x, dither):
    """bf16 bits of fp32 x, `dither` added to the 16 bits that are cut off."""
    bits = np.asarray(x, dtype=np.float32).view(np.uint32)
    out = np.where((bits & 0x7F800000) == 0x7F800000, bits, bits + dither.astype(np.uint32))
    return (out >> np.uint32(16)).astype(np.uint16)
