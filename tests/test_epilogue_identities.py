"""The arithmetic of epilogue.h's erfc, operation by operation in fp32 on the CPU: the
errors that its comment states."""

import os
import re

import numpy as np
from scipy.special import erfc

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "bit_weight_only_quantize_amd", "csrc", "epilogue.h")


def test_erfc_is_as_good_as_it_says():
    f, d = np.float32, np.float64
    text = open(HEADER).read()
    coeffs = [float(x) for x in re.search(r"constexpr float c\[10\] = \{([^}]*)\}", text).group(1).replace("f", "").split(",")]
    z = np.linspace(0, 9.3, 300001).astype(f)
    fma = lambda a, b, c: (a.astype(d) * d(b) + d(c)).astype(f)   # noqa: E731
    t = f(1) / fma(z, f(0.5), f(1))
    p = np.full_like(z, f(coeffs[9]))
    for c in coeffs[8::-1]:
        p = (p.astype(d) * t.astype(d) + d(f(c))).astype(f)
    # e^x as 2^(x log2 e), the product rounded; the power itself is good to an ulp
    power = np.exp2(((-z * z) * f(1.44269504)).astype(d)).astype(f)
    error = np.abs((p * t * power).astype(d) / erfc(z.astype(d)) - 1)
    ulp = 2.0 ** -23
    assert error[z <= 1].max() <= 4.6e-7 + ulp
    assert error[z <= 4].max() <= 1.4e-6 + ulp
    assert error.max() <= 7.9e-6 + ulp
    t64 = 1 / (1 + 0.5 * z.astype(d))
    fit = np.polynomial.polynomial.polyval(t64, [d(f(c)) for c in coeffs]) * t64 * np.exp(-z.astype(d) ** 2)
    assert np.abs(fit / erfc(z.astype(d)) - 1).max() <= 1.8e-7
