"""The two quotients that stand for tanh in the capped scores: the errors that the kernels'
comments state, for the coefficients as the source has them."""
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = np.float32


def numbers(text):
    return [float(x) for x in re.findall(r"(\d+\.\d+(?:e-\d+)?)f", text)]


def source():
    """(p, q) of the quotient for all scores and of the one for small ones, highest degree first."""
    text = open(os.path.join(ROOT, "fp4_kv_cache_rope_gb300", "csrc", "kv8_scores.cuh")).read()
    far = text[text.index("void kv8_tanh_parts"):text.index("// A score over the cap")]
    p, q = (numbers(far[far.index(f"  {x} = "):].split(";")[0]) for x in "pq")
    near = text[text.index("NearCap(float mul"):text.index("one = kv8_pair")]
    at = {m[0]: numbers(m[1])[0] for m in re.findall(r"(p1|p2|q1|q2) = kv8_pair\((.*?),", near)}
    return (p, q), ([at["p2"], at["p1"], 1.0], [at["q2"], at["q1"], 1.0])


FAR, NEAR = source()


def fma(a, b, c):
    """Rounded to fp32 once but for rare ties: a product of fp32 numbers is exact in fp64."""
    return (a.astype(np.float64) * np.asarray(b, np.float64) + np.asarray(c, np.float64)).astype(F)


def horner(c, u, of):
    r = np.full_like(u, of(c[0]))
    for x in c[1:]:
        r = fma(r, u, of(x)) if of is F else r * u + x
    return r


def test_the_source_has_the_coefficients():
    assert [len(x) for x in FAR] == [5, 5] and FAR[0][-1] == FAR[1][-1] == 1.0
    assert FAR[0][-2] == 0.13379715383052826 and NEAR[1][1] == 0.4429476857185364


@pytest.mark.parametrize("which,end,bound", [(FAR, 9.02, 4.3e-8), (NEAR, 2.0, 8.9e-8)])
def test_the_fits(which, end, bound):
    for cast in (float, F):
        y = np.linspace(1e-4, end, 400001)
        p, q = ([float(cast(x)) for x in c] for c in which)
        e = np.abs(y * horner(p, y * y, float) / horner(q, y * y, float) / np.tanh(y) - 1)
        assert 0.95 * bound < e.max() <= bound


def test_the_end():
    """Beyond the end the quotient's value there stands for tanh, which is within half a
    step of 1 in fp32."""
    assert 1 - np.tanh(9.02) < 2.0 ** -25


def test_all_scores_in_fp32():
    y = np.linspace(1e-4, 9.02, 1000001).astype(F)
    u = y * y
    p = horner(FAR[0], u, F) * y
    got = p * (F(1) / horner(FAR[1], u, F))
    e = np.abs(got / np.tanh(y.astype(np.float64)) - 1)
    assert 3e-7 < e.max() < 4e-7 and e.mean() < 6e-8


def test_small_scores_in_fp32():
    """With the factor in the coefficients and two scores to a reciprocal, as the kernel has them."""
    rng, worst = np.random.default_rng(1), 0.0
    (p2, p1, _), (q2, q1, _) = NEAR
    for mul in np.exp(rng.uniform(np.log(1e-6), np.log(1e6), 40)).astype(F):
        m2 = mul * mul
        c = [mul * (m2 * (m2 * F(p2))), mul * (m2 * F(p1)), mul]
        d = [m2 * (m2 * F(q2)), m2 * F(q1), F(1)]
        s = (rng.uniform(1e-4, 2, 200000) / mul).astype(F)
        other = (rng.uniform(-2, 2, 200000) / mul).astype(F)
        n, qa, qb = s * horner(c, s * s, F), horner(d, s * s, F), horner(d, other * other, F)
        got = n * (qb * (F(1) / (qa * qb)))
        x = s.astype(np.float64) * float(mul)
        on = x <= 2
        worst = max(worst, np.abs(got[on] / np.tanh(x[on]) - 1).max())
    assert 3e-7 < worst < 4.5e-7
