"""Binary32 numbers as three bf16 ones, and products of two of them as the output head's
kernels make them, on the CPU; inputs whose results are one product each."""
import numpy as np

U = 2.0 ** -24
PAIRS = ((0, 2), (2, 0), (1, 1), (0, 1), (1, 0), (0, 0))

# A product of two binary32 numbers in six bf16 ones: what is left out is 2^-25 of it at
# most, and each of six additions to a binary32 sum is off by a step at most (half of one,
# if it rounds to the nearest) of the sum so far, which before the last one is less than
# 2^-7 of the product: 0.5 + 2 (1 + 5/128).
PRODUCT = 2.6 * U


def planes(x):
    """Three bf16 numbers, each the nearest to what the ones before leave."""
    rest, out = np.asarray(x, np.float32), []
    for _ in range(3):
        b = rest.view(np.uint32).astype(np.uint64)
        b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
        p = b.astype(np.uint32).view(np.float32)
        out.append(p.astype(np.float64))
        rest = rest - p
    return out


def product(x, y, without=None):
    """The six products' sum, or five's."""
    a, b = planes(x), planes(y)
    return sum(a[i] * b[k] for i, k in PAIRS if (i, k) != without)


def mantissas(rng, *shape):
    """Numbers from 1 to 2 with all their bits."""
    return (1 + rng.random(shape)).astype(np.float32)


def logits_of_one_product(rng, rows, vocab, width):
    """(x, embed, largest logits): each row of x has one element, and each column of embed
    one positive one."""
    k = rng.integers(0, width, rows)
    k[:min(rows, width)] = rng.permutation(width)[:min(rows, width)]
    x = np.zeros((rows, width), np.float32)
    x[np.arange(rows), k] = mantissas(rng, rows)
    embed = -mantissas(rng, vocab, width)
    top = rng.integers(0, vocab, width)
    embed[top, np.arange(width)] = mantissas(rng, width)
    one = x[np.arange(rows), k], embed[top[k], k]
    return x, embed, one


def one_in_each_column(rng, rows, cols, first=0):
    """A matrix with one element in each column, below row `first`, and where they are."""
    at = first + rng.permutation(rows - first)[np.arange(cols) % (rows - first)]
    m = np.zeros((rows, cols), np.float32)
    m[at, np.arange(cols)] = mantissas(rng, cols)
    return m, at


def gradient_error(log_s):
    """Relative, of a * p * e for p = exp(-log_s) of a given log_s: log2(e) and the product
    with it are each off by u of the exponent, the power of two by a step, a's and the result's
    units and their product by u each, and the product of planes."""
    return (2 * log_s + 2 + 3) * U + PRODUCT
