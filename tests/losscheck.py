"""Error bounds of the training-loss kernels against the 64-bit oracle, from
their arithmetic.  U = 2^-24 is half a unit of fp32.

An exponential's base-2 argument a = x c - m carries the rounding of c, of the
difference and of the reference: at most 8 U A over the two arguments a result
depends on, A the largest |a| that matters (2^a below 2^-158, 110 nats, is
nothing) plus 32 (a log-sum-exp exceeds the maximum by at most log2 of the
row's length).  2^a itself is good to 2^-22.  A sum of
positive terms in which one thread adds s terms is good to (s + 32) U.  So a
probability's relative error, and a relative log-sum-exp's absolute one, is at
most ``delta`` below; a loss sum p d with sum p = 1 then moves by at most
delta (2 + sum p |d|), and a gradient entry by delta times the terms it is the
difference of, plus the rounding to its type.
"""

from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
# half a unit in the last place, and half the smallest step, of the types
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -126), torch.bfloat16: (2.0 ** -8, 2.0 ** -126),
         torch.float16: (2.0 ** -11, 2.0 ** -25)}


def f64(t) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def largest(*arrays) -> float:
    """Largest finite magnitude."""
    m = 0.0
    for a in arrays:
        a = np.abs(np.asarray(a, np.float64))
        a = a[np.isfinite(a)]
        if a.size:
            m = max(m, float(a.max()))
    return m


def delta(n: int, span: float) -> float:
    """n entries in a row, span the largest |x| / tau."""
    return 2.0 ** -21 + 8 * U * (min(span, 110.0) / math.log(2) + 32) + (n / 128 + 32) * U


def assert_within(got, want, bound, what: str) -> None:
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bound = np.broadcast_to(np.asarray(bound, np.float64), want.shape)
    assert got.shape == want.shape, f"{what}: shape {got.shape} vs {want.shape}"
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN positions differ"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and not np.isinf(got[~inf]).any(), \
        f"{what}: infinities differ"
    fin = np.isfinite(want)
    err = np.abs(got[fin] - want[fin])
    over = err > bound[fin]
    if over.any():
        i = int(np.argmax(err - bound[fin]))
        raise AssertionError(f"{what}: {int(over.sum())} of {err.size} outside the bound, worst "
                             f"got {got[fin][i]} want {want[fin][i]} bound {bound[fin][i]}")
