"""The attention's calls as programs make them: buffers cut from one allocation,
and what of that is refused. Needs a GB300."""

import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu

BF16, E4M3 = ir.KV_LATENT_BF16, ir.KV_LATENT_E4M3
NOPE, PE, D = 448, 64, 512


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _batch(rows=3, pages=10, page=64, nh=64, fmt=BF16, seed=0):
    """A written cache, queries, page table and ragged lengths."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = ir.kv_latent_empty(rows * pages, page, NOPE, PE, fmt)
    x = torch.randn(rows * pages * page, D, generator=g, device="cuda").to(torch.bfloat16)
    ir.kv_latent_write(cache, x, torch.arange(len(x), dtype=torch.int32, device="cuda"), NOPE, PE)
    q = torch.randn(rows, nh, D, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(rows * pages, generator=g, device="cuda").to(torch.int32).view(rows, pages).contiguous()
    lens = torch.linspace(pages * page, 1, rows, device="cuda").int()
    return q, cache, table, lens


def test_a_workspace_cut_from_one_buffer_with_other_arguments():
    """Behind the workspace's last byte anything may lie; on it nothing may."""
    args = _batch()
    want = ir.latent_attn_decode(*args, NOPE, PE)
    nbytes = ir.latent_attn_workspace_bytes(3, 64, 640, NOPE, PE)
    assert nbytes > 0 and nbytes % 16 == 0  # (a row that is split)
    named = dict(zip(("q", "cache", "table", "lens"), args), O=torch.empty_like(want[0]), lse=torch.empty_like(want[1]))
    for name, t in named.items():
        size = t.numel() * t.element_size()
        begin = -(-size // 16) * 16  # of the workspace
        buffer = torch.zeros(begin + nbytes + size, dtype=torch.uint8, device="cuda")
        ws = buffer[begin:begin + nbytes]
        for at, ok in ((0, True), (16, False), (begin + nbytes - 16, False), (begin + nbytes, True)):
            moved = buffer[at:at + size].view(t.dtype).view(t.shape).copy_(t)
            v = {**named, name: moved}
            call = lambda: ir.latent_attn_decode(v["q"], v["cache"], v["table"], v["lens"], NOPE, PE, O=v["O"],
                                                 lse=v["lse"], workspace=ws)
            if not ok:
                with pytest.raises(ir.InvropeError, match="INVALID"):
                    call()
                continue
            O, lse = call()
            assert torch.equal(O, want[0]) and torch.equal(lse, want[1]), name
