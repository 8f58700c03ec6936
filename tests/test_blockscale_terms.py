"""The block-scale decode's probabilities as the tensor core gets them, modelled in 64 bits:
three e5m2 terms, each of the rest that the ones before leave, 16 times as large. No GPU needed."""
import math

import numpy as np

TARGET, BOUND, SCALE = 12, 15, 16.0


def e5m2(x):
    """Nearest e5m2 number (3 bits, the smallest step 2^-16), ties to even, saturated."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 3, -16))
    return np.clip(np.rint(x / step) * step, -57344.0, 57344.0)


def held(p):
    """The value that the three terms of p stand for."""
    total, rest = np.zeros_like(p), p
    for term in range(3):
        t = e5m2(rest)
        total = total + t / SCALE ** term
        rest = (rest - t) * SCALE
    return total


def test_the_model_of_e5m2():
    import torch
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 2.0 ** np.arange(4000).__mod__(30) / 2 ** 14,
                        [0.0, 2.0 ** -17, 3 * 2.0 ** -17, 2.0 ** -16, 57344.0, 2.5, 3.5, -1.125]])
    t = torch.tensor(x, dtype=torch.float32).clamp(-57344.0, 57344.0)  # torch rounds larger ones to infinity
    assert np.array_equal(e5m2(torch.tensor(x, dtype=torch.float32).numpy()), t.to(torch.float8_e5m2).float().numpy())


def test_products_keep_nine_bits_over_29_octaves_and_eight_over_30():
    rng = np.random.default_rng(1)
    p = np.concatenate([2.0 ** rng.uniform(-14, BOUND, 400000), np.ldexp(1.0, np.arange(-14, BOUND + 1))])
    assert np.all(np.abs(held(p) - p) <= 2.0 ** -9 * p)
    p = 2.0 ** rng.uniform(-15, -14, 100000)
    assert np.all(np.abs(held(p) - p) <= 2.0 ** -8 * p)
    # the largest product is 2^TARGET at least: the stated range is 2^-27 of it
    assert -15 - TARGET == -27


def test_below_that_the_error_is_absolute():
    rng = np.random.default_rng(2)
    p = 2.0 ** rng.uniform(-60, -15, 200000)
    assert np.all(np.abs(held(p) - p) <= 2.0 ** (TARGET - 35))


def test_no_term_saturates():
    p = np.linspace(2.0 ** (BOUND - 2), 2.0 ** BOUND, 30001)
    rest = p
    for _ in range(3):
        t = e5m2(rest)
        rest = (rest - t) * SCALE
        assert np.all(np.abs(rest) <= 2.0 ** BOUND)


def test_the_sum_s_terms_stay_in_fp32():
    """x - m <= spread + bound - target = 83 octaves, and at most 2^30 positions."""
    spread = 80
    assert spread + BOUND - TARGET + 30 + math.log2(2) < 127


# ------------------------------------------------------------------------------ q
def q_terms(q):
    """The value that the three e4m3 terms of a head's elements (bf16 numbers) stand for."""
    from oracle.fp8_block import LUT, encode, needed_scale
    s = needed_scale(q)                      # a power of two
    y = q / s
    hi = LUT[encode(y)]
    mid = LUT[encode(16.0 * (y - hi))]
    lo = LUT[encode(2.0 ** 22 * (y - hi - mid / 16.0))]
    return (hi + mid / 16.0 + lo / 2.0 ** 22) * s


def bf16(x):
    """Nearest bf16 number: 8 bits, and no step below 2^-133."""
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.rint(x / step) * step


def test_q_is_exact_down_to_2_to_the_minus_18_of_its_largest_element():
    rng = np.random.default_rng(3)
    for top in (1.0, 448.0, 449.0, 1.7421875, 3.0e-5, 1.0e30, 2.0 ** -120):
        top = float(bf16(np.array(top)))
        x = bf16(top * 2.0 ** rng.uniform(-18, 0, 50000) * rng.choice([-1.0, 1.0], 50000))
        x = np.append(x[np.abs(x) >= 2.0 ** -18 * top], top)
        assert np.array_equal(q_terms(x), x)


def test_smaller_elements_of_q_are_off_by_2_to_the_minus_25_of_the_largest():
    rng = np.random.default_rng(4)
    x = np.append(bf16(2.0 ** rng.uniform(-60, -18, 100000) * rng.choice([-1.0, 1.0], 100000)), 1.0)
    assert np.all(np.abs(q_terms(x) - x) <= 2.0 ** -25)
