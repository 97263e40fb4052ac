"""Numbers that a C int would cut: the binding hands on none of them as another number.
Needs no GPU."""

import os

import pytest
import torch

import partial_inverse_rope_gb300 as ir
from partial_inverse_rope_gb300 import binding
from partial_inverse_rope_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(binding.lib_path()):
        build()


class _OnDevice(torch.Tensor):
    """A host tensor that says it lies on a GPU."""
    is_cuda = True

    def get_device(self):
        return 0


def _there(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnDevice)


class _Stream:
    cuda_stream, device_index = 0, 0


FAR = 2**32


@pytest.mark.parametrize("nope,pe,fmt", [(FAR + 448, 64, 0), (448, FAR + 64, 1), (448 + FAR, 64 - FAR, 1), (448, 64, FAR), (448, 64, FAR + 4),
                                         (448 - FAR, 64, 4), (FAR**3 + 448, 64, 0)])
def test_no_cache_row(nope, pe, fmt):
    assert ir.kv_latent_row_bytes(nope, pe, fmt) == 0
    with pytest.raises(ValueError, match="no cache row"):
        ir.kv_latent_empty(2, 4, nope, pe, fmt, device="cpu")


@pytest.mark.parametrize("at", range(6))
def test_no_workspace(at):
    args = [8, 64, 4096, 448, 64, 4]
    seen = []

    class Library:
        def invrope_latent_workspace_bytes(self, *a):
            seen.append(a)
            return 0

        def latent_attn_workspace_bytes(self, *a):
            seen.append(a)
            return 0

    args[at] += 2**64 if at in (0, 2) else FAR
    with pytest.MonkeyPatch.context() as m:
        m.setattr(binding, "lib", lambda: Library())
        ir.invrope_latent_workspace_bytes(*args)
        if at < 5:
            ir.latent_attn_workspace_bytes(*args[:5])
    for a in seen:  # what the library gets fits its types, and is not the number that was cut
        assert all(-2**63 <= v < 2**63 if k in (0, 2) else -2**31 <= v < 2**31 for k, v in enumerate(a))
        assert a[at] == (2**63 - 1 if at in (0, 2) else 2**31 - 1)


@pytest.mark.parametrize("nope,pe", [(FAR + 448, 64), (448 + FAR, 64 - FAR), (448, 64 - FAR)])
def test_calls_over_a_cache(monkeypatch, nope, pe):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    i32 = torch.int32
    cache, x, q = _there(2, 4, 512), _there(2, 512), _there(2, 3, 512)
    slots, table, s = _there(2, dtype=i32), _there(2, 2, dtype=i32), _Stream()
    for call in (lambda: ir.kv_latent_write(cache, x, slots, nope, pe, stream=s),
                 lambda: ir.kv_latent_read(cache, slots, nope, pe, out=_there(2, 512), stream=s),
                 lambda: ir.latent_attn_decode(q, cache, table, slots, nope, pe, O=_there(2, 3, 512),
                                               lse=_there(2, 3, dtype=torch.float32), stream=s),
                 lambda: ir.latent_attn_sparse(q, cache, table, nope, pe, O=_there(2, 3, 512),
                                               lse=_there(2, 3, dtype=torch.float32), stream=s)):
        with pytest.raises(ValueError, match="(nope|pe) must be below"):
            call()


@pytest.mark.parametrize("scaling", [FAR + 1, FAR, -FAR, 2**70 + 3])
def test_a_kind_of_scaling(scaling):
    with pytest.raises(ir.InvropeError, match="INVALID_ARG"):
        ir.rope_freqs(64, scaling=scaling, factor=2.0)


def test_more_frequencies_than_an_int_holds(monkeypatch):
    """2^31 + 1 of them are 2^32 + 2 channels, cut to 32 bits two."""
    class Many(torch.Tensor):
        shape = (2**31 + 1,)

    seen = []

    class Library:
        def rope_apply(self, tensors, count, freqs, where, pos0, n, pe, *_):
            seen.append(pe)
            return 2

        def invrope_status_string(self, status):
            return b"UNSUPPORTED"

    monkeypatch.setattr(binding, "lib", lambda: Library())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    freqs = torch.ones(4, dtype=torch.float64).as_subclass(Many)
    with pytest.raises(ir.InvropeError, match="UNSUPPORTED"):
        ir.rope_apply(_there(3, 2, 64), freqs, offset=0, out=_there(3, 2, 64), stream=_Stream())
    assert 512 < seen[0] < 2**31
