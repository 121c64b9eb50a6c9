"""The rotation's angles in wide integers: theta^(-2i/rot) / (2 pi) turns per position to some 60
digits, times a position of any size modulo one turn."""
import decimal
import functools
import math

BITS = 220


@functools.lru_cache(None)
def _pi():
    # Machin: pi / 4 = 4 atan(1/5) - atan(1/239)
    one = 1 << (BITS + 40)

    def atan(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= n * n
            k += 1
        return total
    return 4 * (4 * atan(5) - atan(239))          # in units of 2^-(BITS + 40)


@functools.lru_cache(None)
def turns(theta, rot):
    """Per pair, in units of 2^-BITS turns."""
    with decimal.localcontext() as ctx:
        ctx.prec = 90
        two_pi = 2 * decimal.Decimal(_pi()) / (1 << (BITS + 40))
        ln = decimal.Decimal(theta).ln()
        return [int((-ln * 2 * i / rot).exp() / two_pi * (1 << BITS) + decimal.Decimal("0.5")) for i in range(rot // 2)]


def angle(position, theta, rot, i):
    """Radians in [-pi, pi)."""
    part = position * turns(theta, rot)[i] % (1 << BITS)
    if part >> (BITS - 1):
        part -= 1 << BITS
    return 2 * math.pi * (part / (1 << BITS))
