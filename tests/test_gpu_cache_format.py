"""Calls over a latent cache whose rows are as wide as another format's, through the
compiled calls and without them. Needs a GB300."""

import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built
from partial_inverse_rope_gb300 import binding

pytestmark = pytest.mark.gpu

E4M3, E2M1 = ir.KV_LATENT_E4M3, ir.KV_LATENT_E2M1


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


@pytest.fixture(params=[True, False], ids=["compiled", "binding"])
def way(request, monkeypatch):
    if request.param:
        if binding._calls is None:
            pytest.skip("the compiled calls were not built")
    else:
        monkeypatch.setattr(binding, "_calls", None)


def _calls(cache, nope, pe, **more):
    d, i32 = nope + pe, dict(dtype=torch.int32, device="cuda")
    x = torch.ones(2, d, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(2, 3, d, dtype=torch.bfloat16, device="cuda")
    slots, table, lens = torch.arange(2, **i32), torch.zeros(2, 1, **i32), torch.ones(2, **i32)
    return {
        "write": lambda: ir.kv_latent_write(cache, x, slots, nope, pe, **more),
        "read": lambda: ir.kv_latent_read(cache, slots, nope, pe, **more),
        "decode": lambda: ir.latent_attn_decode(q, cache, table, lens, nope, pe, **more)[0],
        "sparse": lambda: ir.latent_attn_sparse(q, cache, table, nope, pe, **more)[0],
    }


@pytest.mark.parametrize("name", ["write", "read", "decode", "sparse"])
def test_a_cache_is_not_taken_for_another_format(way, name):
    """224 + 64 channels in 8 bits are rows of 368 bytes, as 448 + 64 in 4 bits."""
    for made, fmt, called in (((224, 64), E4M3, (448, 64)), ((448, 64), E2M1, (224, 64))):
        cache = ir.kv_latent_empty(3, 4, *made, fmt)
        cache.zero_()
        with pytest.raises(ValueError, match="rows must be"):
            _calls(cache, *called)[name]()
        assert not cache.any()
        _calls(cache, *made)[name]()


@pytest.mark.parametrize("name", ["write", "read", "decode", "sparse"])
def test_a_call_says_the_format(way, name):
    cache = torch.zeros(3, 4, 368, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="rows must be"):
        _calls(cache, 448, 64, fmt=E4M3)[name]()
    with pytest.raises(ValueError, match="rows must be"):
        _calls(cache, 224, 64, fmt=E2M1)[name]()
    with pytest.raises(ValueError, match="fmt must be"):
        _calls(cache, 448, 64, fmt=3)[name]()
    assert not cache.any()
    got = _calls(cache, 448, 64, fmt=E2M1)[name]()
    assert torch.equal(got, _calls(cache, 448, 64)[name]())
    made = ir.kv_latent_empty(3, 4, 448, 64, E2M1)
    with pytest.raises(ValueError, match="fmt says"):
        _calls(made, 448, 64, fmt=E4M3)[name]()


def test_ordinary_calls_stay_compiled_calls():
    if binding._calls is None:
        pytest.skip("the compiled calls were not built")
    x = torch.ones(2, 512, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(2, dtype=torch.int32, device="cuda")
    for fmt in (ir.KV_LATENT_BF16, E4M3, E2M1):
        made = ir.kv_latent_empty(3, 4, 448, 64, fmt)
        for cache, said in ((made, None), (made, fmt), (made.view(2, 6, -1), None), (made.view(2, 6, -1), fmt)):
            assert binding._calls.latent_write(cache, x, slots, 448, 64, said) is cache
            assert binding._calls.latent_read(cache, slots, 448, 64, said) is not None
