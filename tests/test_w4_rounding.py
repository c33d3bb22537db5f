"""The 4-bit quantizer's quotients: a reciprocal within an ulp, corrected once,
rounds like exact arithmetic for every pair of bf16 significands (ties to even)."""
import numpy as np
import pytest


@pytest.mark.parametrize("ulps", [-1, 0, 1])
def test_corrected_quotient_rounds_exactly(ulps):
    f = np.float32
    sig = np.arange(128, 256).astype(np.float64)
    for m in (np.arange(128, 256) / 256).astype(f):          # the scale's significand in [1/2, 1)
        r = f(1.0 / np.float64(m))
        r = r if ulps == 0 else np.nextafter(r, f(0) if ulps < 0 else f(4))
        for e in range(-14, 6):                               # |v / s| from 2^-14 to past the clamp
            n = (sig * 2.0 ** (e - 7)).astype(f)
            q = n * r
            # a fused multiply-add: float64 holds the product and the difference exactly
            res = (n.astype(np.float64) - q.astype(np.float64) * np.float64(m)).astype(f)
            q = (res.astype(np.float64) * np.float64(r) + q.astype(np.float64)).astype(f)
            assert np.array_equal(np.rint(q), np.rint(n.astype(np.float64) / np.float64(m)))
