"""CPU checks of the polynomials that cap scores of the 4-bit cache's attention: the constants are
read from the source, the errors taken over their ranges, and the coefficients derived
again by the same published method (least maximal relative error, Lawson's iteration)."""
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "block_sparse_flash_attn_gb300", "csrc", "kv4.cuh")
#         name     terms range  error
FITS = [("kTanh", 6, 0.8, 7e-8), ("kNear", 4, 0.3, 2.5e-8)]


def _number(name):
    return float(re.search(name + r" = (-?[0-9.eE+-]+)f", open(SRC).read()).group(1))


def _constants(name, terms):
    return np.array([_number(f"{name}{i}") for i in range(terms)])


def _grid(most):
    return np.linspace(0.0, most, 400_001)[1:]


@pytest.mark.parametrize("name,terms,most,error", FITS)
def test_error_over_the_range(name, terms, most, error):
    assert _number(name + "Range") == most
    y = _grid(most)
    got = np.polynomial.polynomial.polyval(y * y, _constants(name, terms).astype(np.float32).astype(np.float64))
    assert np.abs(got * y / np.tanh(y) - 1.0).max() <= error


@pytest.mark.parametrize("name,terms,most,error", FITS)
def test_fit(name, terms, most, error):
    """The method's own polynomial, at Chebyshev points of y^2, is as good as the constants to within
    their rounding to 32 bits (2^-24 of the first, which is about 1)."""
    u = 0.5 * most * most * (1.0 - np.cos(np.pi * (np.arange(800) + 0.5) / 800))
    y = np.sqrt(u)
    want, w = np.tanh(y) / y, np.full(800, 1.0 / 800)
    powers = (u / (most * most))[:, None] ** np.arange(terms)
    best = np.inf
    for _ in range(300):
        s = np.sqrt(w) / want
        c = np.linalg.lstsq(powers * s[:, None], want * s, rcond=None)[0]
        off = np.abs(powers @ c / want - 1.0)
        best = min(best, off.max())
        w = w * off
        w /= w.sum()
    k = _constants(name, terms)
    mine = np.abs(np.polynomial.polynomial.polyval(u, k) / want - 1.0).max()
    assert mine <= best + 2.0 ** -24 + 2.0 ** -26
