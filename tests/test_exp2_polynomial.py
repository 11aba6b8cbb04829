"""The polynomial that the prompt scores take some exponentials by, on the CPU:
the constants as they stand in the source, float32 steps as the kernel makes
them, against 2^y in 64 bits."""
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_02_b200", "csrc",
                      "prompt_scores.cuh")


@pytest.fixture(scope="module")
def constants():
    text = open(SOURCE).read()
    body = re.search(r"kPsConst\[9\] = \{(.*?)\};", text, re.S).group(1)
    pairs = re.findall(r"\{(-?[0-9.]+)f, (-?[0-9.]+)f\}", body)
    assert len(pairs) == 9 and all(a == b for a, b in pairs)
    return [np.float32(a) for a, _ in pairs]


def rounded(x):
    return x.astype(np.float32).astype(np.float64)


def horner(coefficients, f):
    """Fused float32 steps: a product of two float32 is exact in 64 bits, and so is the sum but for its last bits."""
    e = np.full(f.shape, float(coefficients[0]))
    for c in coefficients[1:]:
        e = rounded(e * f + float(c))
    return e


def test_on_the_reduced_range(constants):
    f = rounded(np.linspace(-0.5, 0.5, 1_000_001))
    exact = np.polyval([float(c) for c in constants[3:]], f) / np.exp2(f) - 1
    assert np.abs(exact).max() <= 1.1e-7
    # float32 steps: under 2^-22, what ex2.approx may be off by
    assert np.abs(horner(constants[3:], f) / np.exp2(f) - 1).max() <= 1.75e-7 < 2.0 ** -22
    assert horner(constants[3:], np.zeros(1))[0] == 1.0


def test_coefficients_are_the_best_of_constant_term_one(constants):
    # no polynomial of degree 5 and constant term 1 is off by less than 9.1e-8 everywhere (a linear program); the
    # coefficients are that one's, rounded to float32
    from scipy.optimize import linprog

    f = 0.5 * np.cos(np.pi * np.arange(1001) / 1000)
    a = np.stack([f ** k for k in (5, 4, 3, 2, 1)], 1) * np.exp2(-f)[:, None]
    b = 1 - np.exp2(-f)
    column = np.full((f.size, 1), -1e-7)  # the bound, in units of 1e-7
    r = linprog([0] * 5 + [1], A_ub=np.block([[a, column], [-a, column]]), b_ub=np.concatenate([b, -b]),
                bounds=[(None, None)] * 5 + [(0, None)], method="highs-ipm",
                options=dict(primal_feasibility_tolerance=1e-10, dual_feasibility_tolerance=1e-10))
    assert 0.90 < r.x[5] < 0.93
    assert np.abs(np.array([float(c) for c in constants[3:8]]) - r.x[:5]).max() < 4e-8


def test_over_all_exponents(constants):
    rng = np.random.default_rng(5)
    y = rounded(np.concatenate([rng.uniform(-128, 128, 400_000), np.arange(-256, 257) / 2.0, [-1e30, 1e30]]))
    c = np.clip(y, -127.0, 127.0)  # clamp_exp2
    t = rounded(c + float(constants[0]))
    n = rounded(t + float(constants[1]))
    f = rounded(n * float(constants[2]) + c)
    assert np.abs(f).max() <= 0.5 and np.array_equal(n + f, c)
    bits = ((t.astype(np.float32).view(np.uint32) << np.uint32(23)) + np.uint32(0x3F800000)).astype(np.uint32)
    power = bits.view(np.float32).astype(np.float64)
    assert np.array_equal(power, np.where(n == -127, 0.0, np.exp2(n)))
    got = horner(constants[3:], f) * power
    assert not got[y <= -127].any()
    some = n > -127
    assert np.abs(got[some] / np.exp2(c[some]) - 1).max() <= 1.75e-7
