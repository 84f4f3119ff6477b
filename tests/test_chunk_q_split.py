"""The two 8-bit parts of a query element in pw_chunk_attn: exact within 2^13 of the row's largest element,
and off by at most what include/pw.h states below.  On every bf16 value of the scaled range (the largest
element of a row lies in [128, 256)), with the formats' rounding taken from ml_dtypes, not from the kernels."""
import ml_dtypes
import numpy as np
import pytest


def _all_bf16_in(lo, hi):
    v = (np.arange(0, 0x8000, dtype=np.uint32) << 16).view(np.float32)
    v = v[np.isfinite(v) & (v >= lo) & (v < hi)]
    return np.concatenate([v, -v])


def _sum_of_parts(x, kind):
    q1 = x.astype(ml_dtypes.float8_e4m3fn).astype(np.float32)
    r = x - q1
    if kind == "e5m2":      # the kernel for many rows
        q2 = r.astype(ml_dtypes.float8_e5m2).astype(np.float64)
    else:                   # the kernel for few
        q2 = (r * np.float32(32)).astype(ml_dtypes.float8_e4m3fn).astype(np.float64) / 32
    assert np.isfinite(q1).all() and np.isfinite(q2).all()
    return q1.astype(np.float64) + q2


@pytest.mark.parametrize("kind", ["e5m2", "e4m3 times 2^5"])
def test_parts_are_exact_within_2_13_of_the_largest(kind):
    x = _all_bf16_in(2.0 ** -6, 256.0)
    assert np.array_equal(_sum_of_parts(x, kind), x.astype(np.float64))


@pytest.mark.parametrize("kind,most", [("e5m2", 2.0 ** -14), ("e4m3 times 2^5", 2.0 ** -15)])
def test_smaller_elements_are_off_by_a_bounded_amount(kind, most):
    x = _all_bf16_in(2.0 ** -100, 2.0 ** -6)
    err = np.abs(_sum_of_parts(x, kind) - x.astype(np.float64))
    assert err.max() == most  # the bound, and it is met
