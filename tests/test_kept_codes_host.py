"""Why the kept activation's codes are those of the exact quotient (CPU only): how near
127 x / m comes to the middle of two codes without being one, x and m any BF16 values.
The kernel's quotient, corrected by its exact remainder, is within 2^-23 of itself, so
2^-17 is far enough."""


def test_no_quotient_is_near_a_half():
    """x = X 2^-e, m = M with 8-bit X, M: |127 X / (M 2^e) - (2 n + 1) / 2| = |254 X - (2 n + 1) M 2^e| / (M 2^(e + 1))
    is compared with 2^-17 of 127 X / (M 2^e) in whole numbers: 2^17 |254 X - (2 n + 1) M 2^e| > 254 X, or 0.  Below a
    quotient of 1/4 (e > 9) every code is 0."""
    nearest = 1.0
    for e in range(10):
        for M in range(128, 256):
            step = M << e
            for X in range(128, 256):
                if X > step:   # x is at most m
                    continue
                whole = 254 * X // step
                for odd in (whole - 1 | 1, whole | 1, whole + 1 | 1):
                    off = abs(254 * X - odd * step)
                    if odd > 0 and off:
                        assert off << 17 > 254 * X, (X, M, e)
                        nearest = min(nearest, off / (2 * step))
    assert 2.0 ** -16 < nearest < 2.0 ** -15
