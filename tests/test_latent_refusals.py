"""Arguments of the latent cache's and attention's calls that are refused on the
host, by the C ABI and by the binding. Needs no GPU."""

import os

import pytest
import torch

from partial_inverse_rope_gb300 import binding
from partial_inverse_rope_gb300.build import build

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA, DEVICE = 0, 1, 2, 3, 4, 5
BF16, E4M3 = 0, 1
A = [k << 40 for k in range(1, 9)]  # far apart, never dereferenced
BIG = 1 << 34


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.lib_path()):
        build()
    return binding.lib()


SHAPE = {"q": A[0], "cache": A[1], "table": A[2], "lens": A[3], "O": A[4], "lse": A[5], "ws": A[6], "nb": BIG,
         "rows": 4, "nh": 64, "nope": 448, "pe": 64, "fmt": BF16, "num_pages": 100, "page": 64, "width": 10,
         "scale": 0.04}


def _decode(lib, **change):
    v = {**SHAPE, **change}
    return lib.latent_attn_decode(v["q"], v["cache"], v["table"], v["lens"], v["O"], v["lse"], v["ws"], v["nb"],
                                  v["rows"], v["nh"], v["nope"], v["pe"], v["fmt"], v["num_pages"], v["page"],
                                  v["width"], v["scale"], None)


def _sparse(lib, **change):
    v = {**SHAPE, **change}
    return lib.latent_attn_sparse(v["q"], v["cache"], v["table"], v["O"], v["lse"], v["ws"], v["nb"], v["rows"],
                                  v["nh"], v["nope"], v["pe"], v["fmt"], v["num_pages"] * v["page"], v["width"],
                                  v["scale"], None)


VEC = 4 * 64 * 512 * 2  # bytes of q and of O


@pytest.mark.parametrize("call,change", [
    (call, change) for call in (_decode, _sparse) for change in (
        {"ws": A[0]}, {"ws": A[0] + VEC - 16}, {"ws": A[0] - 64},        # q
        {"ws": A[1] + 1024}, {"ws": A[1] + 6400 * 1024 - 16},            # cache
        {"ws": A[2], "width": 300}, {"ws": A[2] - 16, "width": 300},     # table
        {"ws": A[4]}, {"ws": A[4] + VEC - 16}, {"ws": A[4] - 1024},      # O
        {"ws": A[5]}, {"ws": A[5] - 16}, {"ws": A[5] + 4 * 64 * 4 - 16},  # lse
    )] + [(_decode, {"ws": A[3], "width": 300}), (_decode, {"ws": A[3] - 16, "width": 300})])
def test_a_workspace_over_another_argument(lib, call, change):
    """Rows that are split: width 10 pages, or 10 or 300 tokens of one page."""
    width = {"width": 640} if call is _sparse and "width" not in change else {}
    assert call(lib, **{**change, **width}) == INVALID


@pytest.mark.parametrize("change", [
    {"ws": A[0] + VEC}, {"ws": A[4] + VEC}, {"ws": A[5] + 4 * 64 * 4}, {"ws": A[1] + 6400 * 1024},
    {"rows": 1, "width": 1, "ws": A[0], "nb": 0},  # one thread block: the workspace is not used
])
def test_a_workspace_beside_them_is_taken(lib, change):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real: only for machines without a GPU")
    assert _decode(lib, **change) in (CUDA, DEVICE)
