"""Pins of the AdamW oracle: torch's AdamW in float64, the level rounding against real
arithmetic, and the random halves."""

import numpy as np
import pytest

from oracle import adamw as A


def test_update_is_torchs_adamw_in_float64():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    p = torch.nn.Parameter(torch.from_numpy(rng.standard_normal(50)))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g)
        opt.step()
        m, v = 0.9 * m + 0.1 * g, 0.95 * v + (1 - 0.95) * g * g
        q, _ = A.update(q, m, v, t, 3e-3, 0.1, 0.9, 0.95, 1e-6)
        assert np.abs(p.detach().numpy() - q).max() < 1e-14


def test_level_is_the_floor_of_the_position_on_the_ladder():
    rng = np.random.default_rng(2)
    x = np.exp(rng.uniform(-60, 60, 4000)).astype(np.float32)
    d = rng.integers(0, 1 << 16, 4000, dtype=np.uint32)
    mant, ex = np.frexp(x.astype(np.float64))
    pos = (ex + 126) * 8 + (2 * mant - 1) * 8                 # exact in float64
    assert np.array_equal(A.levels(x, d), np.floor(pos + d / 65536.0).astype(np.int64))
    # every value of the ladder is a fixed point whatever the dither
    y = A._value(A.levels(x, d))
    assert np.array_equal(A._value(A.levels(y, d)), y)


def test_rounding_is_unbiased_over_the_dither():
    """Over all 2^16 dithers the mean of the rounded value is x to within the 2^-16 of a step
    that the dither resolves, a step being at most 2^-3 of x."""
    d = np.arange(1 << 16, dtype=np.uint32)
    for x in (1.0, 1.03, 1.9, 0.77e-12, 3.3e9):
        y = A._value(A.levels(np.full(1 << 16, x, dtype=np.float32), d)).astype(np.float64)
        assert abs(y.mean() - np.float64(np.float32(x))) <= x * 2.0 ** -3 * 2.0 ** -16 * 1.01
        b = A.cut_bf16(np.full(1 << 16, x, dtype=np.float32), d)
        z = (b.astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)
        assert abs(z.mean() - np.float64(np.float32(x))) <= x * 2.0 ** -7 * 2.0 ** -16 * 1.01


def test_codes_keep_zero_the_top_and_the_window():
    m = np.zeros(600, dtype=np.float32)
    v = np.zeros(600, dtype=np.float32)
    m[:4] = [1.0, -0.5, 2.0 ** -15, 2.0 ** -17]       # the last is below m's 127 levels
    v[:3] = [1.0, 2.0 ** -31, 2.0 ** -40]             # the last is below v's 255 levels
    m[300], v[300] = -3.0, 9.0                        # the second block has its own tops
    z = np.zeros(600, dtype=np.uint32)
    cm, cv, tops = A.encode(m, v, z, z)
    dm, dv = A.decode(cm, cv, tops)
    assert dm[:4].tolist() == [1.0, -0.5, 2.0 ** -15, 0.0]
    assert dv[0] == 1.0 and dv[1] == 2.0 ** -31
    assert 0 < dv[2] < 2.0 ** -31                     # code 1, never 0
    assert dm[300] == -3.0 and dv[300] == 9.0
    assert (cm[4:256] == 0).all() and (cv[3:256] == 0).all() and tops[2] == 0


def test_random_halves_are_uniform_and_uncorrelated():
    """n = 2^18 draws of 16 bits: the mean's standard error is 2^16 / sqrt(12 n) = 37 (five of
    them allowed), a correlation's 1 / sqrt(n) = 0.002 (five of them allowed)."""
    n = 1 << 18
    for seed, step, index in ((0, 1, 0), (12345, 137, 7)):
        sets = A.dithers(seed, step, index, n)
        nxt = A.dithers(seed, step + 1, index, n)
        for i, x in enumerate(sets):
            f = x.astype(np.float64)
            assert abs(f.mean() - 32767.5) < 5 * 37
            assert np.bincount(x >> 12, minlength=16).min() > n / 16 * 0.95
            others = [y for j, y in enumerate(sets) if j != i] + [nxt[i], np.roll(x, 1), np.roll(x, 4)]
            for y in others:
                assert abs(np.corrcoef(f, y.astype(np.float64))[0, 1]) < 5 * 0.002
