"""The latent cache's and attention's C ABI without a GPU: exported symbols, row
sizes, and arguments that are refused on the host before anything is enqueued."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import partial_inverse_rope_gb300 as ir
from oracle import latent_oracle as L
from partial_inverse_rope_gb300 import binding
from partial_inverse_rope_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA, DEVICE = 0, 1, 2, 3, 4, 5
BF16, E4M3 = 0, 1
A = [k << 40 for k in range(1, 9)]  # far apart, never dereferenced
BIG = 1 << 34


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.lib_path()):
        build()
    return binding.lib()


def test_declared_entry_points_are_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "latent_attn.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b((?:kv_latent|latent_attn)_[a-z0-9_]*)\s*\(", text)))
    assert names == ["kv_latent_read", "kv_latent_row_bytes", "kv_latent_write", "latent_attn_decode",
                     "latent_attn_sparse", "latent_attn_workspace_bytes"]
    for n in names:
        assert hasattr(lib, n) and n in binding._SIGNATURES and hasattr(ir, n)


@pytest.mark.parametrize("nope,pe,fmt,want", [
    (448, 64, BF16, 1024), (448, 64, E4M3, 592), (96, 32, E4M3, 176), (48, 16, E4M3, 96), (16, 0, E4M3, 32),
    (0, 8, BF16, 16), (6, 2, BF16, 16), (480, 32, E4M3, 560), (512, 0, E4M3, 528),
    (6, 3, BF16, 0), (0, 0, BF16, 0), (-8, 16, BF16, 0), (8, 8, E4M3, 0), (0, 64, E4M3, 0), (16, 4, E4M3, 0),
    (448, 64, 2, 0), (448, 64, -1, 0), (512, 64, BF16, 0), (2**31 - 8, 8, BF16, 0),
])
def test_row_bytes(lib, nope, pe, fmt, want):
    assert lib.kv_latent_row_bytes(nope, pe, fmt) == want


@pytest.mark.parametrize("change,want", [
    ({"n": -1}, INVALID), ({"num_slots": 0}, INVALID), ({"num_slots": 2**31}, UNSUPPORTED), ({"n": 2**31}, UNSUPPORTED),
    ({"nope": 440, "fmt": E4M3}, INVALID), ({"pe": 4}, INVALID), ({"nope": 512}, UNSUPPORTED), ({"fmt": 7}, INVALID),
    ({"a": None}, INVALID), ({"b": None}, INVALID), ({"c": None}, INVALID),
    ({"a": A[0] + 8}, INVALID), ({"c": A[2] + 8}, INVALID), ({"b": A[1] + 2}, INVALID),
    ({"a": A[2] + 64}, INVALID), ({"b": A[2] + 64}, INVALID),  # inside the cache
    ({"n": 0, "a": None, "b": None, "c": None}, OK),
])
def test_cache_calls_refuse(lib, change, want):
    v = {"a": A[0], "b": A[1], "c": A[2], "n": 8, "num_slots": 64, "nope": 448, "pe": 64, "fmt": BF16, **change}
    tail = (v["n"], v["num_slots"], v["nope"], v["pe"], v["fmt"], None)
    assert lib.kv_latent_write(v["a"], v["b"], v["c"], *tail) == want
    if v["b"] != A[2] + 64:  # a reading call writes neither the cache nor the slots
        assert lib.kv_latent_read(v["c"], v["b"], v["a"], *tail) == want


def test_read_refuses_slots_under_its_output(lib):
    assert lib.kv_latent_read(A[2], A[0] + 64, A[0], 8, 64, 448, 64, BF16, None) == INVALID


DECODE = {"q": A[0], "cache": A[1], "table": A[2], "lens": A[3], "O": A[4], "lse": A[5], "ws": A[6], "nb": BIG,
          "rows": 4, "nh": 64, "nope": 448, "pe": 64, "fmt": BF16, "num_pages": 100, "page": 64, "width": 10,
          "scale": 0.04}


def _decode(lib, **change):
    v = {**DECODE, **change}
    return lib.latent_attn_decode(v["q"], v["cache"], v["table"], v["lens"], v["O"], v["lse"], v["ws"], v["nb"],
                                  v["rows"], v["nh"], v["nope"], v["pe"], v["fmt"], v["num_pages"], v["page"],
                                  v["width"], v["scale"], None)


def _sparse(lib, **change):
    v = {**DECODE, **change}
    return lib.latent_attn_sparse(v["q"], v["cache"], v["table"], v["O"], v["lse"], v["ws"], v["nb"], v["rows"],
                                  v["nh"], v["nope"], v["pe"], v["fmt"], v["num_pages"] * v["page"], v["width"],
                                  v["scale"], None)


BOTH = [
    ({"rows": -1}, INVALID), ({"nh": 0}, INVALID), ({"nh": 129}, UNSUPPORTED), ({"rows": 2**25, "nh": 64}, UNSUPPORTED),
    ({"scale": float("nan")}, INVALID), ({"scale": float("inf")}, INVALID), ({"nope": 450}, INVALID),
    ({"nope": 512}, UNSUPPORTED), ({"nope": 440, "fmt": E4M3}, INVALID), ({"fmt": 3}, INVALID),
    ({"width": -1}, INVALID), ({"width": 2**31}, UNSUPPORTED), ({"num_pages": 0}, INVALID),
    ({"num_pages": 2**31}, UNSUPPORTED),
    ({"q": None}, INVALID), ({"cache": None}, INVALID), ({"table": None}, INVALID), ({"O": None}, INVALID),
    ({"q": A[0] + 8}, INVALID), ({"cache": A[1] + 8}, INVALID), ({"O": A[4] + 2}, INVALID),
    ({"table": A[2] + 1}, INVALID), ({"lse": A[5] + 2}, INVALID),
    ({"O": A[0]}, INVALID), ({"O": A[1] + 1024}, INVALID), ({"lse": A[0] + 64}, INVALID), ({"lse": A[4] + 64}, INVALID),
    ({"rows": 0, "q": None, "cache": None, "table": None, "lens": None, "O": None, "lse": None, "ws": None, "nb": 0}, OK),
]


@pytest.mark.parametrize("change,want", BOTH + [
    ({"lens": None}, INVALID), ({"lens": A[3] + 2}, INVALID), ({"page": 0}, INVALID),
    ({"num_pages": 2**26, "page": 64}, UNSUPPORTED), ({"O": A[3] - 64}, INVALID),
])
def test_decode_refuses(lib, change, want):
    assert _decode(lib, **change) == want


@pytest.mark.parametrize("change,want", BOTH)
def test_sparse_refuses(lib, change, want):
    assert _sparse(lib, **change) == want


@pytest.mark.parametrize("change", [
    {}, {"lse": None}, {"nh": 1}, {"nh": 128}, {"page": 1}, {"page": 48}, {"width": 0}, {"width": 0, "table": None},
    {"fmt": E4M3}, {"nope": 0, "pe": 8}, {"nope": 6, "pe": 2},
])
def test_valid_arguments_reach_the_device_check(lib, change):
    """Without a GPU a valid call stops where it asks for the device."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real: only for machines without a GPU")
    for call in (_decode, _sparse):
        assert call(lib, **change) in (CUDA, DEVICE)


def test_binding_refuses_host_tensors_and_wrong_types():
    cache = torch.zeros(4, 16, 64, dtype=torch.bfloat16)
    x, slots = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ir.kv_latent_write(cache, x, slots, 48, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ir.kv_latent_read(cache, slots, 48, 16)
    with pytest.raises(TypeError):
        ir.kv_latent_read(cache.float(), slots, 48, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ir.latent_attn_decode(torch.zeros(1, 2, 64, dtype=torch.bfloat16), cache,
                              torch.zeros(1, 1, dtype=torch.int32), slots[:1], 48, 16)
    with pytest.raises(TypeError):
        ir.latent_attn_sparse(torch.zeros(1, 2, 64), cache, torch.zeros(1, 4, dtype=torch.int64), 48, 16)
    with pytest.raises(ValueError):
        ir.kv_latent_empty(4, 16, 8, 8, ir.KV_LATENT_E4M3, device="cpu")
    assert ir.kv_latent_empty(4, 16, 48, 16, ir.KV_LATENT_E4M3, device="cpu").shape == (4, 16, 96)
    assert ir.kv_latent_empty(4, 16, 48, 16, device="cpu").dtype == torch.bfloat16


def test_oracle_codes_agree_with_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(L.e4m3_value(codes.numpy()), want, equal_nan=True)
    y = torch.randn(5000, generator=torch.Generator().manual_seed(3), dtype=torch.float64) * 100
    y = torch.cat([y, y.float().half().double() / 64, torch.tensor([448.0, 460.0, 1e9, 0.0, 2.0**-10, 1.5 * 2.0**-9])])
    want = y.clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)
    keep = y.float().double() == y  # torch rounds the fp32 value
    assert np.array_equal(L.e4m3_nearest(y[keep].numpy()), want[keep].numpy())


def test_oracle_attention_is_a_weighted_mean():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((3, 8)), rng.standard_normal((5, 8))
    valid = np.array([True, False, True, True, False])
    O, lse, _, _ = L.attention(q, k, valid, 0.0)  # equal weights
    assert np.allclose(O, k[valid].mean(0)) and np.allclose(lse, np.log(3))
    O, lse, _, _ = L.attention(q, k, np.zeros(5, bool), 1.0)
    assert not O.any() and np.all(lse == -np.inf)
