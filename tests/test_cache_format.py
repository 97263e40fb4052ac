"""The format of a latent cache: what a call says, what the tensor carries, what the width
of a row tells. Needs no GPU."""

import copy
import os

import pytest
import torch

import partial_inverse_rope_gb300 as ir
from partial_inverse_rope_gb300 import binding
from partial_inverse_rope_gb300.build import build

BF16, E4M3, E2M1 = ir.KV_LATENT_BF16, ir.KV_LATENT_E4M3, ir.KV_LATENT_E2M1


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(binding.lib_path()):
        build()


class _OnDevice(torch.Tensor):
    """A host tensor that says it lies on a GPU."""
    is_cuda = True


def _empty(nope, pe, fmt, carries=True):
    t = ir.kv_latent_empty(2, 4, nope, pe, fmt, device="cpu")
    there = t.as_subclass(_OnDevice)
    if carries:
        there.__dict__.update(t.__dict__)
    return there


# splits of one row width, in two formats
SAME = [((224, 64), E4M3, (448, 64), E2M1), ((256, 0), E4M3, (512, 0), E2M1), ((64, 32), E4M3, (96, 40), E2M1)]


@pytest.mark.parametrize("made,fmt,called,other", SAME)
def test_a_cache_is_not_taken_for_another_format(made, fmt, called, other):
    assert ir.kv_latent_row_bytes(*made, fmt) == ir.kv_latent_row_bytes(*called, other) > 0
    cache = _empty(*made, fmt)
    assert binding._cache(cache, *made) == fmt
    with pytest.raises(ValueError, match="rows must be"):  # 8-bit rows under a split that is as wide in 4 bits
        binding._cache(cache, *called)
    cache = _empty(*called, other)
    assert binding._cache(cache, *called) == other
    with pytest.raises(ValueError, match="rows must be"):  # and the other way round
        binding._cache(cache, *made)


@pytest.mark.parametrize("made,fmt,called,other", SAME)
def test_a_call_says_the_format_of_a_tensor_that_carries_none(made, fmt, called, other):
    cache = _empty(*made, fmt, carries=False)
    assert binding._cache(cache, *called) == other  # the width is all there is
    assert binding._cache(cache, *called, other) == other and binding._cache(cache, *made, fmt) == fmt
    with pytest.raises(ValueError, match="rows must be"):
        binding._cache(cache, *called, fmt)
    with pytest.raises(TypeError, match="bfloat16"):
        binding._cache(cache, *made, BF16)


def test_what_a_call_says_has_to_be_what_the_tensor_carries():
    cache = _empty(448, 64, E2M1)
    assert binding._cache(cache, 448, 64, E2M1) == E2M1
    with pytest.raises(ValueError, match="the cache is e2m1, fmt says e4m3"):
        binding._cache(cache, 448, 64, E4M3)
    for fmt in (2, 3, -1, 2**32 + 1, "e2m1", 1.5):
        with pytest.raises(ValueError, match="fmt must be one of"):
            binding._cache(cache, 448, 64, fmt)


@pytest.mark.parametrize("fmt", [BF16, E4M3, E2M1])
def test_views_and_copies(fmt):
    t = ir.kv_latent_empty(2, 4, 448, 64, fmt, device="cpu")
    assert copy.deepcopy(t)._kv_latent_fmt == fmt
    for other in (t.view(1, 8, -1), t[1:], t.clone()):
        assert binding._cache(other.as_subclass(_OnDevice), 448, 64) == fmt


def test_bf16_rows_of_another_split_are_the_same_rows():
    assert binding._cache(_empty(448, 64, BF16), 480, 32) == BF16
    assert binding._cache(_empty(448, 64, BF16), 480, 32, BF16) == BF16
