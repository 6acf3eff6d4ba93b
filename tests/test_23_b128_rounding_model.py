"""The arithmetic by which the block-128 quantize rounds x / s without dividing, replayed in numpy FP32 against exact
fractions (CPU): 1/s moved to the side that s was rounded away from, one product, its low 8 bits cut off.

With X and A the 8-bit mantissas of x and of the block's largest element, x / s is next to the middle of two codes only
where 7 X 2^k = A o for the middle's odd factor o <= 31, and otherwise at least 1 / (255 * 31) away from it, so every
pair of mantissas at every distance of exponents settles the claim for all inputs."""
from fractions import Fraction

import numpy as np
import pytest

MIDS = np.array([(2 * i + 1) / 2 ** 10 for i in range(8)]
                + [(2 * m + 17) / 16 * 2.0 ** e for e in range(-6, 9) for m in range(8)])[:126]
VALUES = np.array([i / 2 ** 9 for i in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)])[:127]


def cast(v):
    """E4M3 code of positive numbers (ties to even), saturating."""
    return np.where(v > 464, 126, np.searchsorted(MIDS, v) + (np.isin(v, MIDS) & (np.searchsorted(MIDS, v) % 2 == 1)))


def exact_code(x, s):
    """Code of the exact quotient x / s."""
    q = Fraction(x) / Fraction(s)
    i = int(np.searchsorted(MIDS, float(q)))
    for j in (i - 1, i):   # the float of the quotient may have crossed one middle
        if 0 <= j < 126:
            m = Fraction(float(MIDS[j]))
            if q == m:
                return j + (j % 2)
    i = sum(1 for j in range(max(i - 2, 0), min(i + 2, 126)) if q > Fraction(float(MIDS[j]))) + max(i - 2, 0)
    return min(i, 126)


def test_tables():
    assert VALUES[126] == 448 and len(MIDS) == 126
    assert np.array_equal(MIDS, (VALUES[1:127] + VALUES[:126]) / 2)


@pytest.mark.parametrize("ulp", [-1, 0, 1])
def test_moved_reciprocal_rounds_as_the_quotient(ulp):
    """`ulp`: the approximate reciprocal's own error."""
    near = 0
    for A in range(128, 256):
        s = np.float32(np.float64(A) * (1.0 / 448.0))
        assert abs(Fraction(float(s)) - Fraction(A, 448)) <= Fraction(float(np.spacing(s))) / 2
        e = Fraction(A) - 448 * Fraction(float(s))
        r = (np.float32(1.0 / np.float64(s)).view(np.int32) + ulp + (516 if e > 0 else -508 if e < 0 else 4)).view(np.float32)
        x = (np.arange(128, 256)[:, None] * 2.0 ** -np.arange(0, 23)[None]).astype(np.float32)
        x = x[x <= A]
        v = ((x * r).view(np.uint32) & np.uint32(0xFFFFFF00)).view(np.float32).astype(np.float64)
        got = cast(v)
        q = x.astype(np.float64) / np.float64(s)
        # where the FP64 quotient is clear of every middle its code is certain
        i = np.searchsorted(MIDS, q)
        d = np.minimum(np.abs(q / MIDS[np.minimum(i, 125)] - 1), np.abs(q / MIDS[np.maximum(i - 1, 0)] - 1))
        clear = d > 1e-9
        assert np.array_equal(got[clear], np.minimum(i[clear], 126))
        assert d[(d > 1e-6)].min() > 1 / 7906     # nothing between a tie and 1 / (255 * 31)
        for j in np.flatnonzero(~clear):
            near += 1
            assert got[j] == exact_code(float(x[j]), float(s)), (A, x[j])
    assert near > 300
