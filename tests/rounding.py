"""bfloat16 rounding in 64 bits, for tests of bfloat16 outputs.

A bfloat16 has 8 bits of significand (7 stored), so a value x in
[2^e, 2^(e+1)) is rounded to a multiple of 2^(e-7), off by at most 2^(e-8)."""
import numpy as np


def quantum(x):
    """Spacing of bfloat16 numbers at x (2^-133 below the normal range)."""
    _, e = np.frexp(np.abs(x))
    return np.ldexp(1.0, np.maximum(e - 8, -133))


def to_bf16(x):
    """x rounded to the nearest bfloat16 (ties to even), as float64."""
    q = quantum(x)
    return np.rint(x / q) * q


def within(got, want, tol, bf16):
    """True where got is `want` up to tol or, with bf16, where got is the
    rounding of a value that is."""
    if not bf16:
        return np.abs(got - want) <= tol
    return (to_bf16(want - tol) <= got) & (got <= to_bf16(want + tol))
