"""CPU check of the software exp2 of the keys' weights: its coefficients are the degree-5 polynomial through
2^f at the six Chebyshev nodes of [-1/2, 1/2], and, evaluated as the kernel does (fp32 Horner after the
round-to-nearest split x = n + f), it stays within 5e-7 relative error of 2^x."""
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_114_b200", "csrc", "evict.cuh")


def coefficients():
    text = open(SRC, encoding="utf-8").read()
    return np.array([float(re.search(rf"kKeyExp2C{i} = ([0-9.eE+-]+)f", text).group(1)) for i in range(6)], np.float32)


def test_coefficients_are_the_interpolant():
    t = 0.5 * np.cos((2 * np.arange(6) + 1) * np.pi / 12)
    c = np.linalg.solve(np.vander(t, 6, increasing=True), np.exp2(t))
    # within one fp32 step of the solved values (the system is solved in fp64)
    assert np.all(np.abs(c - coefficients()) <= np.spacing(coefficients()))
    # interpolation error: max |(2^t)^(6)| / (6! 2^5) (1/2)^6
    f = np.linspace(-0.5, 0.5, 100_001)
    assert np.abs(np.polyval(c[::-1], f) - np.exp2(f)).max() <= np.log(2) ** 6 * np.sqrt(2) / (720 * 32 * 64)


def test_relative_error():
    c, magic = coefficients(), np.float32(12582912.0)
    x = np.linspace(-125.0, 1.0, 2_000_001).astype(np.float32)
    t = (x + magic).astype(np.float32)
    f = (x - (t - magic).astype(np.float32)).astype(np.float32)
    q = c[5]
    for k in range(4, -1, -1):
        q = (q * f + c[k]).astype(np.float32)
    y = (q.view(np.int32) + (t.view(np.int32) << 23)).astype(np.int32).view(np.float32).astype(np.float64)
    # interpolation 1.1e-7 (absolute, so at most 1.6e-7 relative), Horner's last two roundings 2 x 2^-24
    # each of values up to sqrt(2) on results from 1 / sqrt(2), and the rounded coefficients: below 5e-7
    assert np.abs(y / np.exp2(x.astype(np.float64)) - 1.0).max() <= 5e-7


def as_the_kernel(x):
    """fp32 Horner after the split, 2^n as a factor (n + 127) << 23; x held at -127, a NaN kept."""
    c, magic = coefficients(), np.float32(12582912.0)
    x = np.where(np.isnan(x), x, np.maximum(x, np.float32(-127.0))).astype(np.float32)
    t = (x + magic).astype(np.float32)
    f = (x - (t - magic).astype(np.float32)).astype(np.float32)
    q = c[5]
    for k in range(4, -1, -1):
        q = (q * f + c[k]).astype(np.float32)
    return q * ((t.view(np.int32) << 23) + np.int32(0x3F800000)).astype(np.int32).view(np.float32)


def test_below_the_smallest_normal_and_not_a_number():
    y = as_the_kernel(np.array([-np.inf, -1e30, -1000.0, -127.0, -126.51], np.float32))
    assert not y.any()
    assert np.isnan(as_the_kernel(np.array([np.nan], np.float32))).all()
    x = np.linspace(-126.0, 1.0, 1_000_001).astype(np.float32)
    y = as_the_kernel(x).astype(np.float64)
    normal = x >= -125.5   # (below, a result may be under 2^-126, which the GPU may take for 0)
    assert np.abs(y / np.exp2(x.astype(np.float64)) - 1.0)[normal].max() <= 5e-7
    # the source holds x at the same place and keeps a NaN
    text = open(SRC, encoding="utf-8").read()
    assert text.count("fmax_nan(x.x, -127.f)") == 1 and text.count("fmax_nan(x.y, -127.f)") == 1
