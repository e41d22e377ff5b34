"""Fits the polynomials of the projections' gelu (gemm.cuh).

gelu(z) = max(z, 0) - t Q(t) with t = |z| and Q(t) = erfc(t / sqrt 2) / 2.  Q is
e^(-t^2/2) R(t) where R(t) = erfcx(t / sqrt 2) / 2 falls from 1/2 as 0.4 / t: with
k = 1 / (1 + c t), R = k P(k) for a smooth P on all of 0 < k <= 1.  What counts
is Q's relative error, because for z < 0 it is the result's.  The coefficients
minimise the largest |R - k P(k)| / R over a grid up to t = 14 (beyond 13.2 the
exponential is below the smallest normal fp32), a linear programme; they are
rounded to fp32 and checked with an fp32 evaluation.

    python fit_gelu_poly.py [degree c]
"""
import sys

import numpy as np
from scipy.optimize import linprog
from scipy.special import erfcx

T_MAX = 14.0


def fit(deg, c):
    t = np.linspace(0, T_MAX, 3000)
    r = 0.5 * erfcx(t / np.sqrt(2))
    k = 1 / (1 + c * t)
    # a basis on [-1, 1] keeps the programme well scaled
    v = np.polynomial.chebyshev.chebvander(2 * k - 1, deg) * (k / r)[:, None]
    one = np.ones((len(t), 1))
    s = linprog(np.r_[np.zeros(deg + 1), 1], A_ub=np.block([[v, -one], [-v, -one]]),
                b_ub=np.r_[one[:, 0], -one[:, 0]],
                bounds=[(None, None)] * (deg + 1) + [(0, None)], method="highs")
    p = np.polynomial.Chebyshev(s.x[:-1], domain=[0, 1]).convert(kind=np.polynomial.Polynomial)
    return np.float32(p.coef), s.x[-1]


def check(coef, c):
    """Largest relative error of R with every operation rounded to fp32."""
    f = np.float32
    t = np.linspace(0, T_MAX, 200001).astype(f)
    k = f(1) / (f(1) + (f(c) * t).astype(f))
    p = np.full(t.shape, coef[-1], f)
    for a in coef[-2::-1]:
        p = (p.astype(np.float64) * k + np.float64(a)).astype(f)
    r = 0.5 * erfcx(t.astype(np.float64) / np.sqrt(2))
    return np.abs((p * k).astype(np.float64) / r - 1).max()


def main():
    # the packed forward's and the fp32 one's
    pairs = [(int(sys.argv[1]), float(sys.argv[2]))] if len(sys.argv) > 2 else [(5, 0.31), (7, 0.3)]
    for deg, c in pairs:
        coef, err = fit(deg, c)
        print(f"degree {deg}, c = {c:g}: relative error {err:.1e}, in fp32 {check(coef, c):.1e}")
        for i, a in enumerate(coef):
            print(f"  k^{i}: {a:.9g}")


if __name__ == "__main__":
    main()
