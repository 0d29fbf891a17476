"""fp32 operands as bf16 planes: what each product may lose, and operands that show
whether the last plane is there.

x = x0 + x1 + x2, each plane what the ones before leave, rounded to bf16: |x1| <= 2^-8
|x|, |x2| <= 2^-16 |x|, and three hold all 24 bits.  A row with a single entry
makes a result one product x y, without a sum in which roundings could hide a
missing plane.  U = 2^-24 is half a step of fp32.  The matrix instructions' sums are not
rounded to the nearest but down, by up to a whole step, 2 U: of x = 2.023238182067871 and
y = -0.51025390625 the five products of three planes by two add up to -1.0323652066290379,
between -1.0323652029037476 and -1.0323653221130371; the device gives the latter.
  three planes by three: the pairs (1, 2), (2, 1) and (2, 2) are left out, at most
      2 U + 2^-8 U of x y; the six others are exact in fp32, and of their five sums
      the last loses 2 U, those before it are 2^-7 of x y: less than U / 8.
  three by two (a 4-bit weight is whole in two): (2, 1) is left out, U; the sums
      as above.
With two planes of x the third is missing: up to 2^-16 |x| = 256 U, 40 U in the mean."""
import numpy as np

from input_adaptive_rank_amd import synth

U = 2.0 ** -24
THREE_BY_THREE, THREE_BY_TWO = 4.2, 3.2   # units of U
PAIRS = {(3, 3): [(2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)], (3, 2): [(2, 0), (1, 1), (1, 0), (0, 1), (0, 0)]}


def planes(x, count):
    out, rest = [], np.asarray(x, dtype=np.float64)
    for _ in range(count):
        out.append(synth.round_bf16(rest))
        rest = rest - out[-1]
    return out


def product(x, y, kind=(3, 3), missing_x=False, missing_y=False):
    """x y as the pairs of planes give it, summed in fp32, smallest first; missing:
    without the last plane of x or y (the planted mistake)."""
    px, py = planes(x, kind[0]), planes(y, kind[1])
    if missing_x:
        px[-1] = 0 * px[-1]
    if missing_y:
        py[-1] = 0 * py[-1]
    acc = np.float32(0)
    for a, b in PAIRS[kind]:
        acc = np.float32(acc + (px[a] * py[b]).astype(np.float32))
    return acc.astype(np.float64)


def numbers(shape, seed):
    """fp32 numbers of all 24 bits."""
    return synth.round_f32(np.random.default_rng(seed).standard_normal(shape) + 3.0)


def single_entries(n, c, seed):
    """[n][c] with one entry a row, in column row mod c; and these entries."""
    x = numbers(n, seed)
    out = np.zeros((n, c))
    out[np.arange(n), np.arange(n) % c] = x
    return out, x


def probability_bound(v):
    """Relative error of p = exp(-lse), lse = log v, of d = w p and of a gradient
    d x, in units of U: the exponent log2 v is a product with a rounded constant (two
    roundings of it, ln 2 of each in p), the power 2, the weights' quotient, two
    products with them, the planes' product, the result."""
    return 2 * np.log(v) + 2 + 3 + THREE_BY_THREE + 1
