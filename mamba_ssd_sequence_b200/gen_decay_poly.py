"""Generates the coefficients of the polynomial q with 1 - exp(-t) ~ t q(t)
on [-1/2, 1/2] that the gated linear recurrence (csrc/ssd_glr.cuh, exact_decay)
uses: Chebyshev interpolation of (1 - exp(-t)) / t at the degree + 1 Chebyshev
nodes, converted to powers of t and rounded to float32.  Prints the
coefficients (constant term first) and the largest relative error of t q(t)
against 1 - exp(-t), evaluated by float32 Horner steps.

    python -m mamba_ssd_sequence_b200.gen_decay_poly [degree]
"""
import sys

import numpy as np


def _exact(t):
    t = np.asarray(t, dtype=np.float64)
    return np.where(t == 0, 1.0, -np.expm1(-t) / np.where(t == 0, 1.0, t))


def coefficients(degree: int = 5) -> np.ndarray:
    k = np.arange(degree + 1)
    n = np.cos((2 * k + 1) * np.pi / (2 * (degree + 1)))  # nodes on [-1, 1]
    cheb = np.polynomial.chebyshev.chebfit(n, _exact(n / 2), degree)
    poly = np.polynomial.Chebyshev(cheb, domain=[-0.5, 0.5]).convert(kind=np.polynomial.Polynomial)
    return poly.coef.astype(np.float32)


def max_rel_error(c32: np.ndarray) -> float:
    t = np.linspace(-0.5, 0.5, 2_000_001)
    x = t.astype(np.float32)
    acc = np.full_like(x, c32[-1])
    for c in c32[-2::-1]:
        acc = (acc * x + c).astype(np.float32)
    return float(np.max(np.abs(acc.astype(np.float64) / _exact(x) - 1)))


if __name__ == "__main__":
    c = coefficients(int(sys.argv[1]) if len(sys.argv) > 1 else 5)
    print(", ".join(f"{v:.9e}f" for v in c))
    print("max relative error:", max_rel_error(c))
