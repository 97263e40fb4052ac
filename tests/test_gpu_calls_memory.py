"""Compiled calls that find no memory for their outputs raise what torch raises, and the next
call is as before. The process keeps itself to a part of the memory. Needs a GB300."""

import gc

import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built
from partial_inverse_rope_gb300 import binding

pytestmark = pytest.mark.gpu


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


def _cases():
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = ir.kv_latent_empty(4, 64, 448, 64, ir.KV_LATENT_E4M3)
    cache.zero_()
    many = 1 << 16  # 64 MB of vectors
    slots = torch.zeros(many, **i32)
    x = torch.zeros(many, 512, dtype=torch.bfloat16, device="cuda")
    q = x.view(1024, 64, 512)
    table = torch.zeros(1024, 1, **i32)
    state, pages, queue = ir.kv_pages_empty(2, 8, 16)
    freqs, _ = ir.rope_freqs(64)
    idx = torch.zeros(1 << 14, 1 << 10, **i32)
    return {
        "read": lambda: ir.kv_latent_read(cache, slots, 448, 64),
        "decode": lambda: ir.latent_attn_decode(q, cache, table, table[:, 0].contiguous(), 448, 64),
        "sparse": lambda: ir.latent_attn_sparse(q, cache, table, 448, 64),
        "rope": lambda: ir.rope_apply(x, freqs),
        "slots": lambda: ir.kv_idx_local_to_slots(idx, pages, state[:2], 4, 16, 1 << 13),
        "pages": lambda: ir.kv_pages_advance(state, pages, queue, state[:2].clone(), 4, 1 << 24),
    }


@pytest.mark.parametrize("name", ["read", "decode", "sparse", "rope", "slots", "pages"])
def test_no_memory_for_the_outputs(way, name):
    call = _cases()[name]
    call()
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    # what is held now and 16 MB more: outputs take 64 MB at least
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (16 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    call()
    torch.cuda.synchronize()
