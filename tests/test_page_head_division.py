"""The page_head store divides by a block's scale through its reciprocal and one residual correction
(csrc/store_page_head.cu).  That gives RN(x / s + e), |e| < 2^-45 x / s, for RN(x / s).  The two differ
only where x / s lies within e of a midpoint between neighbouring floats, and the codes only where one
of those neighbours is a border between codes.

e: y = RN(1/s) = (1 + d1) / s, q = RN(x y) = x/s (1 + d), |d| <= 2^-23 + 2^-47; the residual q s - x = x d
is fused and rounded by 2^-24, times y by 2^-24 more: the corrected quotient is x/s (1 - d d4) with
|d4| < 2^-22.4, so |e| < 2^-45 x/s before its own rounding."""
import numpy as np


def _solutions(mid, most):
    """Normalised (8-bit odd part of x, 24-bit s, n) with x 2^k = s * mid + n, |n| <= most."""
    found = []
    for n in range(-most, most + 1):
        # x has 8 bits, so the left side has at least this many trailing zeros
        zeros = max(0, (mid << 23).bit_length() - 1 - 8)
        step = 1 << zeros
        s = (-n * pow(mid, -1, step)) % step
        while s < 1 << 24:
            v = s * mid + n
            if s >= 1 << 23 and v > 0:
                odd = v >> ((v & -v).bit_length() - 1)
                if odd < 256:
                    found.append((odd, s, n))
            s += step
    return found


def test_no_quotient_is_close_enough_to_a_midpoint_beside_a_code_border():
    """Borders have at most 9 significant bits B; the midpoints beside one are B 2^16 +- 1 in units of
    half a float's step (below a power of two, half that).  |x/s - mid| = |n| / s half steps, and e is
    below 2^-45 * 2^25 = 2^-20 of them, so |n| < 2^24 * 2^-20 = 16."""
    found = []
    for B in range(256, 512):
        found += _solutions(B * 2 ** 16 + 1, 16) + _solutions(B * 2 ** 16 - 1, 16)
    found += _solutions(256 * 2 ** 17 - 1, 32)
    # the one that there is: every bit of s set, x a power of two; the kernel divides plainly then
    assert found == [(1, 2 ** 24 - 1, 1)]


def _e4m3_borders():
    return sorted({(2 * n + 1) * 2.0 ** -10 for n in range(8)} |
                  {(16 + 2 * m + 1) * 2.0 ** (e - 4) for e in range(-6, 9) for m in range(8)})


def test_borders_have_at_most_nine_bits():
    for b in _e4m3_borders() + [n + 0.5 for n in range(127)]:
        m = np.frexp(b)[0] * 2 ** 9
        assert m == int(m)
