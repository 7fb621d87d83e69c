"""Generate gated_poly.cuh: polynomials of the gated linear recurrence's coefficients in y = 2 v, v the
decay exponent, on [0, 1/4] (v up to 1/8).

  e^{-y/2}                  ~= 1 + y P(y)     the decay a
  sqrt((1 - e^{-y}) / y)    ~= 1 + y P(y)     g: the input weight sqrt(1 - a^2) is sqrt(y) g
  1 / g                     ~= 1 + y P(y)     v / sqrt(1 - a^2) is sqrt(y) / (2 g)

Fitted in fp64 by least squares on Chebyshev nodes, reweighted towards the largest residuals, to the
function less 1 over y, so that the polynomials are exact at 0.

Run:  python gen_gated_poly.py > gated_poly.cuh
The errors of the fp32 Horner evaluation, relative to the function, are printed beside each.
"""
import numpy as np

TOP = 0.25


def fit(f, deg, n=4000, iters=60):
    k = np.arange(n)
    x = TOP * (np.cos(np.pi * (k + 0.5) / n) + 1) / 2
    V = np.vander(x, deg + 1, increasing=True)
    t = (f(x) - 1) / x
    weight = x / f(x)  # the error that counts is x P - (f - 1), relative to f
    w = weight.copy()
    best = None
    for _ in range(iters):
        c, *_ = np.linalg.lstsq(V * w[:, None], t * w, rcond=None)
        r = np.abs((V @ c - t) * weight)
        if best is None or r.max() < best[0]:
            best = r.max(), c
        w = w * (1 + 2 * r / r.max())
        w /= w.max()
    return best[1]


def error(f, c):
    x = np.linspace(1e-7, TOP, 1000001).astype(np.float32)
    p = np.float32(c[-1])
    for ci in c[-2::-1]:
        p = np.float32(p * x.astype(np.float64) + np.float64(np.float32(ci)))
    v = np.float32(p.astype(np.float64) * x + 1)
    return np.abs(v - f(x.astype(np.float64))).max() / f(TOP)


def main():
    g = lambda y: np.sqrt(-np.expm1(-y) / y)  # noqa: E731
    print("// generated by gen_gated_poly.py -- do not edit by hand")
    print("#pragma once")
    for name, f, deg in (("DECAY", lambda y: np.exp(-y / 2), 3), ("WEIGHT", g, 2), ("WEIGHT_INV", lambda y: 1 / g(y), 2)):
        c = fit(f, deg)
        print(f"// max relative error of the fp32 evaluation {error(f, c):.2e}")
        print(f"#define SSM_GATED_{name}_POLY {{" + ", ".join(f"{float(np.float32(v))!r}f" for v in c) + "}")


if __name__ == "__main__":
    main()
