"""2 pi to more bits than any angle of the tests needs."""
from fractions import Fraction


def circle():
    """2 pi as a fraction, off by less than 2^-400 (Machin: pi = 16 atan(1/5) - 4 atan(1/239))."""
    one = 1 << 420

    def atan(d):
        total, term, i = 0, one // d, 1
        while term:
            total += term // i if i % 4 == 1 else -(term // i)
            term //= d * d
            i += 2
        return total

    return Fraction(2 * (16 * atan(5) - 4 * atan(239)), one)
