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

    |silu'| <= 1.1, so g's own error dg gives 1.1 dg.  For a given g, the
    exponential of -g is off by at most 3 U from the function and (2 |g| + 1) U
    from its argument's scaling to base 2, which reach silu times a factor
    below 1; the addition, the reciprocal (2 U) and two multiplies add 5 U."""
    g, u = product(a, sa, *gate), product(a, sa, *up)
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    dg, du = 3.1 * U * np.abs(g), 3.1 * U * np.abs(u)
    ds = 1.1 * dg + np.abs(s) * (2 * np.abs(g) + 9) * U
    return s * u, 1.01 * (np.abs(u) * ds + np.abs(s) * du) + np.abs(u) * 2.0 ** -118


def groups(offsets) -> list[tuple[int, int, int]]:
    """(expert, first row, past the last row) of the groups that have rows."""
    o = [int(v) for v in offsets]
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def tolerance(y: np.ndarray, bound: np.ndarray, t: str) -> np.ndarray:
    """Half a step of the output's type at the largest value y may have come to, beside the bound."""
    smallest = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[t]     # half a subnormal step
    return bound + HALF_EPS[t] * (np.abs(y) + bound) + smallest
