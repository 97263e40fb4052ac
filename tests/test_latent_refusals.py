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


@pytest.mark.parametrize("call", [_decode, _sparse])
@pytest.mark.parametrize("scale,want", [
    (2.4e38, INVALID), (-2.4e38, INVALID), (1e300, INVALID), (float("nan"), INVALID), (float("-inf"), INVALID),
    (2.3e38, None), (-2.3e38, None), (1e-320, None), (0.0, None),
])
def test_a_scale_beyond_fp32(lib, call, scale, want):
    """It would make an infinity of every score, and NaN of a score of zero."""
    if want is None and torch.cuda.is_available():
        pytest.skip("the addresses are not real: only for machines without a GPU")
    st = call(lib, scale=scale)
    assert st == want if want is not None else st in (CUDA, DEVICE)


@pytest.mark.parametrize("nh", [1, 3, 64, 127, 128])
def test_the_most_rows(lib, nh):
    """rows * nh < 2^31: with the most rows a call gets as far as its addresses."""
    most = (2**31 - 1) // nh
    for call in (_decode, _sparse):
        assert call(lib, rows=most, nh=nh, width=1, q=None) == INVALID
        assert call(lib, rows=most + 1, nh=nh, width=1, q=None) == UNSUPPORTED


class _OnDevice(torch.Tensor):
    """A host tensor that says it lies on a GPU."""
    is_cuda = True

    def get_device(self):
        return self.index


def _there(index, *shape, dtype=torch.bfloat16):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(_OnDevice)
    t.index = index
    return t


class _Stream:
    cuda_stream = 0

    def __init__(self, index):
        self.device_index = index


class _Library:
    """Stands for the library: no entry point may be called but the size queries."""

    def kv_latent_row_bytes(self, nope, pe, fmt):
        return 2 * (nope + pe)

    def latent_attn_workspace_bytes(self, *_):
        return 0


def _calls(index, other=None, stream=None):
    """The four calls with their tensors on `index`, and `other` for one in the
    name's place."""
    on = lambda name, *shape, **k: _there(other[1] if other and other[0] == name else index, *shape, **k)
    i32 = torch.int32
    cache = lambda: on("cache", 4, 16, 64)
    q = lambda: on("q", 2, 3, 64)
    out = lambda: {"O": on("O", 2, 3, 64), "lse": on("lse", 2, 3, dtype=torch.float32)}
    return {
        "write": lambda: binding.kv_latent_write(cache(), on("x", 2, 64), on("slots", 2, dtype=i32), 48, 16,
                                                 stream=stream),
        "read": lambda: binding.kv_latent_read(cache(), on("slots", 2, dtype=i32), 48, 16, out=on("out", 2, 64),
                                               stream=stream),
        "decode": lambda: binding.latent_attn_decode(q(), cache(), on("table", 2, 4, dtype=i32),
                                                     on("lens", 2, dtype=i32), 48, 16, stream=stream, **out()),
        "sparse": lambda: binding.latent_attn_sparse(q(), cache(), on("table", 2, 4, dtype=i32), 48, 16, stream=stream,
                                                     **out()),
    }


@pytest.fixture
def two_devices(monkeypatch):
    monkeypatch.setattr(binding, "lib", lambda: _Library())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda index: pytest.fail("no call changes the current device"))
    binding._row_width.cache_clear()
    binding._workspace_bytes.cache_clear()
    yield
    binding._row_width.cache_clear()
    binding._workspace_bytes.cache_clear()


@pytest.mark.parametrize("name", ["write", "read", "decode", "sparse"])
def test_binding_refuses_tensors_and_streams_of_a_device_that_is_not_current(two_devices, name):
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        _calls(1)[name]()
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        _calls(1, stream=_Stream(1))[name]()
    with pytest.raises(ValueError, match="stream must be of cuda:0, got cuda:1"):
        _calls(0, stream=_Stream(1))[name]()


@pytest.mark.parametrize("name,args", [("write", ["cache", "x", "slots"]), ("read", ["cache", "slots", "out"]),
                                       ("decode", ["cache", "q", "table", "lens", "O", "lse"]),
                                       ("sparse", ["cache", "q", "table", "O", "lse"])])
def test_binding_refuses_one_tensor_of_another_device(two_devices, name, args):
    for arg in args:
        with pytest.raises(ValueError, match="cuda:"):
            _calls(0, other=(arg, 1), stream=_Stream(0))[name]()


@pytest.mark.parametrize("name", ["write", "read", "decode", "sparse"])
def test_binding_calls_the_library_with_tensors_of_the_current_device(two_devices, name):
    with pytest.raises(AttributeError, match=name):  # the stand-in has no entry point
        _calls(0, stream=_Stream(0))[name]()
