"""The corrected quotient (tests/test_markstein_quotient.py) on numerators with
all 24 bits, as the rotary append has them: rotated keys are fp32. An e4m3 code
depends on the quotient through the boundaries between codes alone, numbers of
at most five significant bits; away from them a quotient within two ulps has the
code of the exact one. So what has to hold is that for numerators within a few
ulps of boundary * scale the corrected quotient is the IEEE one. Exponents change
nothing while nothing over- or underflows, so significands are all there is: all
2^23 of a scale's with all 16 of a boundary's and 17 numerators about their
product were compared with fmaf in C (2 281 701 376 quotients, no difference);
here a sample of the scales, at several exponents."""
import numpy as np

from test_markstein_quotient import _corrected


def test_quotients_next_to_every_code_boundary():
    rng = np.random.default_rng(3)
    m = (np.arange(16, 32) / 16).astype(np.float64)
    sig = np.unique(np.concatenate([np.arange(0, 1 << 23, 1 << 13), rng.integers(0, 1 << 23, 600), [1, 2, 3, (1 << 23) - 1, (1 << 23) - 2]]))
    checked = 0
    for i in sig:
        e = int(rng.integers(-79, 60))
        s = np.float32(np.ldexp(1 + int(i) * 2.0 ** -23, e))
        k = int(rng.integers(-9, 9))                                  # e4m3 values: 2^-9 to 448
        x0 = np.ldexp(m * float(s), k).astype(np.float32)             # RN(boundary * scale)
        x = (x0.view(np.int32)[:, None] + np.arange(-8, 9, dtype=np.int32)).astype(np.int32).view(np.float32).ravel()
        x = np.concatenate([x, -x])
        q, y = _corrected(x, s)
        assert np.all(np.abs(x).astype(np.float64) * abs(float(y)) < 2.0 ** 100)
        with np.errstate(all="ignore"):
            assert np.array_equal(q, x / s), float(s)
        checked += x.size
    assert checked > 800_000


def test_quotients_of_random_fp32_numerators():
    rng = np.random.default_rng(5)
    for s in np.concatenate([np.float32(2.0) ** rng.uniform(-30, 30, 150).astype(np.float32), np.nextafter(np.float32([0.25, 1, 8]), np.float32(0)),
                             np.nextafter(np.float32([0.25, 1, 8]), np.float32(9))]):
        x = (s * np.float32(2.0) ** rng.uniform(-11, 9, 8000).astype(np.float32)).astype(np.float32)
        q, _ = _corrected(x, np.float32(s))
        assert np.array_equal(q, x / np.float32(s)), float(s)
