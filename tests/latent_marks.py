"""Values for attention tests that show the loss of a few tokens of a long row.

With ordinary values a token's share of the output shrinks with the row's length,
while the tolerance, which adds up all weights' roundings, does not: a lost tile
of 64 tokens can pass. Here a channel is non-zero in few tokens, and so is what the
tolerance allows there: the tokens of a tile (``per="tile"``), or every d-th token
(``per="token"``)."""

import numpy as np


def marked(n, d, per):
    """float64 [n, d]: 1 in one channel of each token, 0 in the others."""
    t = np.arange(n)
    x = np.zeros((n, d))
    x[t, (t // 64 if per == "tile" else t) % d] = 1.0
    return x
