"""Fit the polynomials used for 2^f on the FMA pipes and write exp2_poly.cuh (the
cubic of the forward) and exp2_poly5.cuh (degree 5, for sums kept in fp32).

    python tiled_attention_24_b200/csrc/fit_exp2_poly.py

The softmax evaluates 2^x as 2^n * p(f) with n = rint(x), f = x - n in
[-1/2, 1/2] and p a degree-3 polynomial ("FlashAttention 4" page, section
"Software exponent on CUDA cores": a cubic evaluated on the FMA units to take
load off the special-function unit).  The coefficients are our own: a minimax
fit of the RELATIVE error, by the Remez exchange algorithm (E. Remez, 1934;
see e.g. Muller, "Elementary Functions", ch. 3), then rounded to fp32 and
re-checked.  bf16 P needs a relative error below 2^-9; the script prints the
maximum relative error of the fp32-rounded coefficients and records it in
the header it writes (7.5e-5, about 2^-13.7).
"""
from __future__ import annotations

import os

import numpy as np

LO, HI, DEG = -0.5, 0.5, 3


def remez(deg=DEG, lo=LO, hi=HI, iters=30):
    n = deg + 2
    # Chebyshev-like initial reference
    k = np.arange(n)
    x = 0.5 * (lo + hi) + 0.5 * (hi - lo) * np.cos(np.pi * (n - 1 - k) / (n - 1))
    grid = np.linspace(lo, hi, 200001)
    for _ in range(iters):
        # p(x_i) - 2^x_i = (-1)^i E 2^x_i   (relative error equioscillates)
        A = np.zeros((n, n))
        for i in range(n):
            A[i, :deg + 1] = x[i] ** np.arange(deg + 1)
            A[i, deg + 1] = -((-1) ** i) * 2.0 ** x[i]
        sol = np.linalg.solve(A, 2.0 ** x)
        c = sol[:deg + 1]
        err = (np.polyval(c[::-1], grid) - 2.0 ** grid) / 2.0 ** grid
        # new reference: one extremum per sign run
        sgn = np.sign(err)
        idx, start = [], 0
        for j in range(1, len(grid) + 1):
            if j == len(grid) or sgn[j] != sgn[start]:
                seg = slice(start, j)
                idx.append(start + int(np.argmax(np.abs(err[seg]))))
                start = j
        if len(idx) < n:
            break
        idx = np.array(idx)
        # keep the n consecutive extrema with the largest minimum magnitude
        best = max(range(len(idx) - n + 1), key=lambda s: np.abs(err[idx[s:s + n]]).min())
        x = grid[idx[best:best + n]]
    return c


def fp32_eval(c32, f):
    """Horner in fp32 with fused multiply-adds (fp64 product+sum, one rounding)."""
    p = np.float32(c32[3])
    for k in (2, 1, 0):
        p = np.float32(np.float64(p) * np.float64(f) + np.float64(c32[k]))
    return p


def main():
    c = remez()
    c32 = np.array(c, dtype=np.float32)
    f = np.linspace(LO, HI, 100001).astype(np.float32)
    p = np.array([fp32_eval(c32, x) for x in f], dtype=np.float64)
    rel = np.abs(p / 2.0 ** f.astype(np.float64) - 1.0).max()
    out = os.path.join(os.path.dirname(os.path.abspath(__file__)), "exp2_poly.cuh")
    with open(out, "w") as fh:
        fh.write("// Generated by fit_exp2_poly.py (minimax cubic for 2^f, f in [-1/2, 1/2],\n")
        fh.write(f"// relative error {rel:.3e} after rounding to fp32).  Do not edit by hand.\n")
        fh.write("#pragma once\n")
        fh.write("namespace ta {\n")
        for k in range(4):
            fh.write(f"constexpr float kExp2C{k} = {float(c32[k]).hex()}f;  // {float(c32[k]):.9g}\n")
        fh.write(f"constexpr float kExp2PolyRelErr = {rel:.6e}f;\n")
        fh.write("}  // namespace ta\n")
    print(out, c32, rel)
    write_degree5()


def write_degree5():
    """Degree 5: as accurate as the hardware exponential (2 ulp), for the weights of a
    prompt's keys, whose probabilities are summed in fp32 and never rounded."""
    c32 = np.array(remez(deg=5), dtype=np.float32)
    f = np.linspace(LO, HI, 100001).astype(np.float32).astype(np.float64)
    p = np.full_like(f, float(c32[5])).astype(np.float32)
    for k in range(4, -1, -1):
        p = (p.astype(np.float64) * f + float(c32[k])).astype(np.float32)
    rel = np.abs(p.astype(np.float64) / 2.0 ** f - 1.0).max()
    out = os.path.join(os.path.dirname(os.path.abspath(__file__)), "exp2_poly5.cuh")
    with open(out, "w") as fh:
        fh.write("// Generated by fit_exp2_poly.py (minimax degree 5 for 2^f, f in [-1/2, 1/2],\n")
        fh.write(f"// relative error {rel:.3e} after rounding to fp32).  Do not edit by hand.\n")
        fh.write("#pragma once\n")
        fh.write("namespace ta {\n")
        for k in range(6):
            fh.write(f"constexpr float kExp2P5C{k} = {float(c32[k]).hex()}f;  // {float(c32[k]):.9g}\n")
        fh.write(f"constexpr float kExp2Poly5RelErr = {rel:.6e}f;\n")
        fh.write("}  // namespace ta\n")
    print(out, c32, rel)


if __name__ == "__main__":
    main()
