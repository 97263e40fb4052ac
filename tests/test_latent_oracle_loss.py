"""What the attention's tolerances let pass: tokens left out of the second product
(their weights still in the sum), as by a stage overwritten early, a tile skipped or
a lost partial. The mistake is planted in the oracle; no GPU."""

import numpy as np
import pytest

from latent_marks import marked
from oracle import latent_oracle as L

D, NH = 512, 3


def _beyond(q, values, lost):
    """How far the output without tokens `lost` is off, in tolerances, at most."""
    n = len(values)
    O, _, tol, _ = L.attention(q, values, np.ones(n, bool), D ** -0.5)
    s = D ** -0.5 * (q @ values.T)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    p[:, lost] = 0
    return float((np.abs(p @ values - O) / np.maximum(tol, 1e-300)).max())


def _queries(size):
    return size * np.random.default_rng(1).standard_normal((NH, D))


@pytest.mark.parametrize("size", [0.0, 0.5])
@pytest.mark.parametrize("n", [700, 9000, 12345, 20011])
def test_marked_values_show_a_lost_tile_and_a_lost_token(n, size):
    q = _queries(size)
    for begin in (0, 64 * (n // 128), 64 * (n // 64)):
        tile = np.arange(begin, min(n, begin + 64))
        assert _beyond(q, marked(n, D, "tile"), tile) > 20
        assert _beyond(q, marked(n, D, "token"), tile) > 1.5
        assert _beyond(q, marked(n, D, "tile"), tile[:4]) > 1.5
        assert _beyond(q, marked(n, D, "token"), tile[:1]) > 1.5


@pytest.mark.parametrize("size", [0.0, 0.5])
def test_marked_values_show_a_lost_tile_of_a_row_over_the_whole_card(size):
    tile = np.arange(32768, 32832)
    assert _beyond(_queries(size), marked(65536, D, "tile"), tile) > 10


def test_ordinary_values_do_not():
    """Why the marked ones: a tile of 20011 normal tokens may go missing unseen."""
    values = np.random.default_rng(2).standard_normal((20011, D))
    assert _beyond(_queries(1.0), values, np.arange(640, 704)) < 1
