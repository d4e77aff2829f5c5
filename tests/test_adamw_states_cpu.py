"""8-bit AdamW states by their definition: what random rounding does to the moments,
and that the second moment's root never becomes zero by it."""

import numpy as np
import pytest

from oracle import fp8_oracle as Q

ALL = np.arange(1 << 20)           # every random number


@pytest.mark.parametrize("r", [0.3, 17.3, 2.0 ** -6, 0.7 * 2.0 ** -6, 3.4 * 2.0 ** -9])
def test_the_root_keeps_its_mean_and_its_square_gains_the_variance(r):
    """r between the neighbours lo and hi: the mean of the stored values is r (within one
    part in 2^20 of the step), that of their squares r^2 + (hi - r)(r - lo)."""
    x = np.zeros(ALL.size)
    x[:] = r
    x[::128] = 300.0               # the block's scale is 1
    q = np.delete(Q.quant_random(x, ALL, True)[0], np.s_[::128])
    lo, hi = q.min(), q.max()
    # numbers 0, 128, 256, ... are the largest values', so the rest are a little uneven:
    # by at most one in 128 of the step's variance
    step = max(hi - lo, r * 2.0 ** -4)
    assert abs(q.mean() - r) <= step / 128
    assert abs((q * q).mean() - r * r - (hi - r) * (r - lo)) <= 2 * hi * step / 128


def test_the_least_value_is_kept_where_it_divides():
    x = np.zeros(256)
    x[0], x[1:5] = 300.0, [1e-3, 1e-5, 1e-12, 1e-30]
    rnd = np.zeros(256, np.int64)
    q, _ = Q.quant_random(x, rnd, True)
    assert (q[1:5] == 2.0 ** -9).all() and (q[5:] == 0).all()
    assert (Q.quant_random(x, rnd)[0][1:] == 0).all()


@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-5, 1e-6])
def test_steps_stay_bounded(size, beta2):
    """Random gradients, half of each block ``size`` times the other half.

    With m = beta1 m_q + (1 - beta1) g and v = beta2 v_q + (1 - beta2) g^2, a step is at most
    |m_q| beta1 / sqrt(beta2 v_q) + (1 - beta1) / sqrt(1 - beta2), the bias corrections aside.  The first
    part: of the largest elements |m| <= c sqrt(v) with c = (1 - beta1) / sqrt((1 - beta2)(1 - beta1^2 /
    beta2)) by Cauchy, 1.16 or 7.3, so the scale of m is at most 2 c that of v; a small m_q rounded up
    every time stands at 1 / (1 - beta1) = 10 of its least values, 20 c of those of sqrt(v), which
    is one at least: 23.2 + 0.4 or 146 + 3.2.  Without the least value: 600 to 1100."""
    n, b1 = 128 * 32, 0.9
    small = np.arange(n) % 128 >= 64
    scale = np.where(small, size, 1.0)
    rng = np.random.default_rng(3)
    m, v, worst = np.zeros(n), np.zeros(n), 0.0
    c = (1 - b1) / np.sqrt((1 - beta2) * (1 - b1 * b1 / beta2))
    most = 20 * c * b1 / np.sqrt(beta2) + (1 - b1) / np.sqrt(1 - beta2)
    for t in range(1, 301):
        _, m, v = Q.adamw(np.zeros(n), rng.normal(size=n) * scale, m, v, 1.0, b1, beta2, 1e-8, 0.0, t)
        step = np.abs(m / (1 - b1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + 1e-8)
        assert step.max() <= most * max(1.0, np.sqrt(1 - beta2 ** t) / (1 - b1 ** t)), t
        out = []
        for x, r, least in zip((m, np.sqrt(v)), Q.random_bits(n, 0, 9, t), (False, True)):
            q, byte = Q.quant_random(x, r, least)
            out.append(q * np.repeat(np.ldexp(1.0, byte - 127), 128))
        m, v = out[0], out[1] ** 2
