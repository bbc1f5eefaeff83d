"""64-bit oracle of the 8-bit operators (quant_i8, gemm_i8 and their SwiGLU
and grouped forms), in numpy.  Shares no code with the HIP path.

The integer sums are exact: float64 holds every integer below 2^53, and the
sums stay below 2^31.  Every bound returned with a result counts the fp32
roundings the header allows before the last one (each at most 2^-24 of the
rounded value); tolerance() adds the rounding to the output's type.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24                                      # half an ulp of fp32, relative
HALF_EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def quant(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(codes int8, scales float32) of x [M, K] (float64 values of the inputs)."""
    x = np.asarray(x, dtype=np.float64)
    codes = np.zeros(x.shape, dtype=np.int8)
    scales = np.empty(x.shape[0], dtype=np.float32)
    for m, row in enumerate(x):
        if not np.isfinite(row).all():
            scales[m] = np.nan
            continue
        s = np.float32(max(np.max(np.abs(row)) / 127.0, 2.0 ** -126))
        scales[m] = s
        # The quotient of two fp32 values is never within 2^-53 of a tie it
        # is not equal to, so rint of the float64 quotient is exact.
        codes[m] = np.rint(row / np.float64(s)).astype(np.int8)
    return codes, scales


def product(a, sa, w, sw) -> np.ndarray:
    """P[m, n] in float64."""
    acc = a.astype(np.float64) @ w.astype(np.float64).T
    return acc * sa.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]


def gemm(a, sa, w, sw, bias=None) -> tuple[np.ndarray, np.ndarray]:
    """(y, bound): the conversion and two multiplies of P, and the addition."""
    p = product(a, sa, w, sw)
    bound = 3.1 * U * np.abs(p)
    if bias is None:
        return p, bound
    y = p + bias.astype(np.float64)[None, :]
    return y, bound + 1.1 * U * np.abs(y)


def swiglu(a, sa, gate, up) -> tuple[np.ndarray, np.ndarray]:
    """(y, bound) of silu(g) * u.

    With c = 1 / (1 + e^g), the weight of a relative error of e^-g in silu(g) =
    g / (1 + e^-g):
    - g's own error dg reaches silu times silu'(g) = (1 + g c) / (1 + e^-g), and in
      the second order times at most e^-|g| (2 + |g|) / 2;
    - the exponential is off by 2 |g| U from its argument's scaling to base 2 and
      by 4 U from the function, taken whole or as the product of two halves,
      times c;
    - its addition to 1 and the reciprocal add 3 U, the products 4 U.
    An exponential below the normal numbers, past |g| = 174.6, may be taken as
    zero, which leaves out less than |u| 2^-244; a product of two small values
    may be subnormal on the way."""
    g, u = product(a, sa, *gate), product(a, sa, *up)
    with np.errstate(over="ignore", invalid="ignore"):
        sig, c, size = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g)), np.abs(g)
        s = g / (1.0 + np.exp(-g))
        dg, du = 3.1 * U * size, 3.1 * U * np.abs(u)
        ds = sig * np.abs(1.0 + g * c) * dg + 0.51 * dg * dg * np.exp(-size) * (2 + size)
        ds += np.abs(s) * ((2 * size + 4) * c + 7) * U
        return s * u, 1.01 * (np.abs(u) * ds + np.abs(s) * du) + np.abs(u) * (size > 174) * 2.0 ** -244 + 2.0 ** -150


def groups(offsets) -> list[tuple[int, int, int]]:
    """(expert, first row, past the last row) of the groups that have rows."""
    o = [int(v) for v in offsets]
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def tolerance(y: np.ndarray, bound: np.ndarray, t: str) -> np.ndarray:
    """Half a step of the output's type at the largest value y may have come to, beside the bound."""
    smallest = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[t]     # half a subnormal step
    return bound + HALF_EPS[t] * (np.abs(y) + bound) + smallest
