"""How far fp32 attention may be off, by norm: the root mean square of its roundings.

u = 2^-24 is the largest relative error of one rounding.  A rounding is taken as
independent of the others and uniform over half a step either way, the values it rounds as
spread evenly over a binade's logarithm: R = u sqrt(3 / (8 ln 2)) / sqrt 3 = 0.425 u of its
result (root mean square).  n terms of random sign added one after another: the partial
sums grow as the root of their number, so the sum is off by R sqrt(n / 2) of its own size;
n terms of one sign by R sqrt(n / 3).  An output's norm is over thousands of elements, so
its error lies near the root mean square; the bounds are twice that (uneven weights, terms
that are dependent), and a last rounding.
"""
import math

U = 2.0 ** -24
R = U * math.sqrt(1.0 / (8.0 * math.log(2.0)))
LN2 = math.log(2.0)


def chain(n):
    """Relative error of n terms of random sign added one after another."""
    return R * math.sqrt(n / 2.0)


def dot(D):
    """Of a product over D columns in two lanes that are joined."""
    return math.sqrt(chain(D / 2) ** 2 + R ** 2)


def scores(D, z):
    """Relative error of a softmax weight by its score's (the product, the scale, the
    maximum taken off), z the scores' root mean square in base 2; the heavy weights have
    scores of about three times that."""
    return LN2 * 3.0 * z * math.sqrt(dot(D) ** 2 + 2 * R ** 2)


def forward(n, D, z):
    """o over n states: 64 of them a tile, folded into the sum so far every eight tiles."""
    tiles = math.ceil(n / 64)
    l = R * math.sqrt(tiles / 3.0 + 6)
    parts = [scores(D, z), 2 * U, l, chain(min(n, 512)), chain(math.ceil(tiles / 8)), R]
    return 2 * math.sqrt(sum(p * p for p in parts)) + U


def weight(D, z, lse):
    """A weight rebuilt as 2^(z - lse): three roundings at lse's size, and ex2's."""
    at_lse = 2.0 ** math.floor(math.log2(max(1.0, abs(lse)))) * U / math.sqrt(3.0)
    return math.sqrt((LN2 * at_lse) ** 2 * 3 + scores(D, z) ** 2 + (2 * U) ** 2)


def gradient(n, D, z, lse):
    """dq over n states, or dk, dv over n rows: 64 a tile, the tiles' sums added up."""
    parts = [weight(D, z, lse), dot(D), R, chain(min(n, 64)), chain(math.ceil(n / 64)), R]
    return 2 * math.sqrt(sum(p * p for p in parts)) + U


LOST = 2.0 ** -15  # an operand rounded to 13 significant bits: 2^-13 / sqrt 12 of it and more
