"""Fits the polynomial of the projections' gelu (gemm.cuh).

gelu(z) = max(z, 0) - t Q(t) with t = |z| and Q(t) = erfc(t / sqrt 2) / 2.  Q is
e^(-t^2/2) R(t) where R(t) = erfcx(t / sqrt 2) / 2 falls slowly from 1/2, so on
[0, 6] a polynomial in t takes R's place (beyond, Q is below 1e-9).  The error
that counts is Q's: relative where Q is large, absolute where it vanishes.
The coefficients minimise the largest |R - p| e^(-t^2/2) / (2^-12 Q + 1e-7)
over a grid, a linear programme; the result is rounded to fp32 and checked
with an fp32 Horner evaluation.

    python fit_gelu_poly.py [degree]
"""
import sys

import numpy as np
from scipy.optimize import linprog
from scipy.special import erfc, erfcx

T_MAX = 6.0


def fit(deg):
    t = np.linspace(0, T_MAX, 1500)
    e = np.exp(-t * t / 2)
    r = 0.5 * erfcx(t / np.sqrt(2))
    tol = np.minimum((1e-7 + 2.0 ** -12 * e * r) / e, 0.25 * r)
    v = np.vander(2 * t / T_MAX, deg + 1, increasing=True)
    a = np.block([[v, -tol[:, None]], [-v, -tol[:, None]]])
    s = linprog(np.r_[np.zeros(deg + 1), 1], A_ub=a, b_ub=np.concatenate([r, -r]),
                bounds=[(None, None)] * (deg + 1) + [(0, None)], method="highs")
    return np.float32(s.x[:-1] / (T_MAX / 2) ** np.arange(deg + 1)), s.x[-1]


def main():
    deg = int(sys.argv[1]) if len(sys.argv) > 1 else 9
    c, factor = fit(deg)
    t = np.linspace(0, T_MAX, 60001)
    p = np.full(t.shape, c[-1], np.float32)
    for k in c[-2::-1]:
        p = np.float32(p.astype(np.float64) * np.float32(t) + np.float64(k))
    q = 0.5 * erfc(t / np.sqrt(2))
    d = np.abs(p * np.exp(-t * t / 2) - q)
    print(f"degree {deg}: |dQ| <= {factor:.3f} (2^-12 Q + 1e-7); in fp32 largest |dQ| {d.max():.2e}, "
          f"|dQ| / Q {(d / q)[t <= 4].max():.1e} up to t = 4, {(d / q)[t <= 5].max():.1e} up to 5")
    for i, k in enumerate(c):
        print(f"c{i} = {k:.9g}")


if __name__ == "__main__":
    main()
