"""``run_decode``'s pool of pages: its size. Needs no GPU."""

import numpy as np
import pytest

from oracle import pages_oracle as P
from partial_inverse_rope_gb300 import run_decode


def _lens(rows, prompt):
    return [int(n) for n in np.linspace(max(1, prompt // 2), prompt, rows, dtype=np.float32)]


@pytest.mark.parametrize("rows,prompt,steps,page", [(5, 300, 6, 64), (1, 1, 0, 64), (3, 200, 3, 64), (8, 4096, 16, 64), (33, 65, 5, 64),
                                                    (7, 129, 1, 128), (2, 64, 60, 16), (64, 1000, 100, 48), (4, 5, 3, 1)])
def test_every_prompt_fits(rows, prompt, steps, page):
    """The pool's own arithmetic: prompts, and the first step after them."""
    lens, most = _lens(rows, prompt), prompt + steps + 4
    pages, width = run_decode.pool_pages(lens, most, page), -(-most // page)
    state = np.array([0] * rows + [0, pages], np.int32)
    got = P.advance(state, np.full((rows, width), -1, np.int32), np.arange(pages, dtype=np.int32), lens, page, sum(lens))
    assert got["granted"].tolist() == lens
    got = P.advance(got["state"], got["table"], got["queue"], [1] * rows, page, rows)
    assert got["granted"].tolist() == [1] * rows


def test_three_quarters_of_what_the_sequences_could_fill():
    assert run_decode.pool_pages(_lens(32, 16384), 16384 + 64 + 4, 64) == 3 * 32 * 258 // 4
