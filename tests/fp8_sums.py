"""Inputs and bounds that show a lost, doubled or misscaled block of an FP8
product at any number of columns.

Whole numbers.  x in -3 .. 3 and w in -2 .. 2, every block of w times 1, 2 or 4
by turns: a value has two significant bits, so quantising changes none, and any
partial sum is a whole number of at most 24 K <= 24 * 65536 < 2^21, which fp32
(and 24-bit significands in the tensor core) hold exactly.  Whatever the order
of the sums, the result is the exact one, rounded once to the output's type.

Random numbers.  A chain of accumulations is at most 16 blocks and three more
where its range starts inside a chunk: 76 steps of 32 columns.  Each adds to an
accumulator that is truncated, a loss of half a unit of its 24-bit significand
on the average, 2^-24 of it, always towards zero.  Over many outputs the
accumulator is nowhere larger, in the 2-norm, than where its chain ends; the
chains' losses are in proportion to the chains, and the sums of chains round to
nearest, with errors of either sign.  So the relative error in the 2-norm stays
below 76 * 2^-24 = 4.5e-6 at any K.
"""
import numpy as np

BLOCK = 128
CHAIN_ERROR = 76 * 2.0 ** -24


def whole(rng, n, k, tokens):
    """(x [tokens][k], w [n][k]) of whole numbers, as fp32."""
    x = rng.integers(-3, 4, (tokens, k)).astype(np.float32)
    w = rng.integers(-2, 3, (n, k)).astype(np.float32)
    return x, w * np.exp2((np.arange(k) // BLOCK) % 3).astype(np.float32)


def one_block(rng, n, k, blocks):
    """The same with token t's values in block blocks[t] alone."""
    x, w = whole(rng, n, k, len(blocks))
    return np.where((np.arange(k) // BLOCK)[None, :] == np.asarray(blocks)[:, None], x, 0).astype(np.float32), w


def relative_error(y, want):
    return float(np.linalg.norm(np.asarray(y, np.float64) - want) / np.linalg.norm(want))
