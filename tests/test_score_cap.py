"""The polynomial of the prefill's score cap, evaluated on the CPU from the coefficients in its
source: cap tanh(x / cap) for scores up to 0.7 of the cap."""
import os
import re

import numpy as np
import pytest

from rank_compressed_paged_gb300 import build


def source():
    with open(os.path.join(build.CSRC, "scoremod.cuh")) as f:
        return f.read()


def coefficients():
    c = [float(x) for x in re.findall(r"c[1-4] = (-?[\d.]+)f(?: \* i2)+;", source())]
    assert len(c) == 4
    return c


def fma(a, b, c):
    """One rounding to fp32 (the fp64 product of two fp32 numbers is exact; the sum's rounding to
    53 bits first is off by 2^-29 of a step at most)."""
    return (a.astype(np.float64) * b + c).astype(np.float32)


def errors(u, y):
    want = np.tanh(u.astype(np.float64))
    err = np.abs(y - want)
    return (err / want).max(), err.max()


def stated():
    """The relative errors of the polynomial and of its fp32 evaluation, and the absolute one, that
    the comment above it gives."""
    text = " ".join(re.sub(r"//", "", source()).split())
    m = re.search(r"relative error ([\d.]+e-7), in fp32 arithmetic ([\d.]+e-7); absolute ([\d.]+e-7) of the cap",
                  text)
    return [float(x) for x in m.groups()]


def test_polynomial_is_as_good_as_its_comment_says():
    u = np.linspace(1e-6, 0.7, 2_000_001)
    v = u * u
    c1, c2, c3, c4 = coefficients()
    rel, absolute = errors(u, u + u * v * (c1 + v * (c2 + v * (c3 + v * c4))))
    exact, _, of_cap = stated()
    assert 0.95 * exact < rel <= exact and absolute <= of_cap


@pytest.mark.parametrize("softcap", [2.0 ** -10, 0.3, 1.0, 15.0, 30.0, 50.0, 1024.0])
def test_its_fp32_evaluation_at_every_cap(softcap):
    """As the kernel does it: in powers of x^2 with the cap in the coefficients, log2 units."""
    f = np.float32
    cap2, inv = f(softcap * np.log2(np.e)), f(1.0 / (softcap * np.log2(np.e)))
    k = [f(c) for c in coefficients()]
    for n in range(4):
        for _ in range(n + 1):
            k[n] = f(k[n] * f(inv * inv))
    x = (np.linspace(1e-6, 0.7, 500_001) * float(cap2)).astype(f)
    w = x * x
    x, w = x[w <= f(0.49) * cap2 * cap2], w[w <= f(0.49) * cap2 * cap2]
    y = fma(x * w, fma(fma(fma(np.full_like(w, k[3]), w, k[2]), w, k[1]), w, k[0]), x)
    assert np.all(np.isfinite(y))
    rel, absolute = errors(x.astype(np.float64) / float(cap2), y.astype(np.float64) / float(cap2))
    assert rel <= stated()[1] and absolute <= stated()[2], (rel, absolute)
