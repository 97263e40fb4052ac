"""The attention's calls as programs make them: buffers cut from one allocation
(and what of that is refused), several rows of one sequence, large caches, several
host threads. Needs a GB300."""

import threading

import numpy as np
import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built, f64
from oracle import latent_oracle as L

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


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_several_new_tokens_of_one_sequence(fmt):
    """Each is a row of its own: the sequence's page list again, with its own length."""
    page, nh, chunk = 16, 20, 5
    cache = ir.kv_latent_empty(200, page, NOPE, PE, fmt)
    slots = torch.arange(200 * page, dtype=torch.int32, device="cuda")
    x = torch.randn(200 * page, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    ir.kv_latent_write(cache, x.cuda(), slots, NOPE, PE)
    values = f64(ir.kv_latent_read(cache, slots, NOPE, PE))
    order = torch.randperm(200, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    last = [3, chunk, 130, 2400]  # tokens of each sequence, its chunk's newest among them
    table = torch.full((len(last), 150), -1, dtype=torch.int32)
    for r in range(len(last)):
        n = -(-last[r] // page)
        table[r, :n] = order[sum(-(-k // page) for k in last[:r]):][:n]
    rows = table.repeat_interleave(chunk, 0).cuda()
    lens = torch.tensor([n - chunk + 1 + k for n in last for k in range(chunk)], dtype=torch.int32)  # 0 and less: no token
    q = torch.randn(len(lens), nh, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    O, lse = ir.latent_attn_decode(q.cuda(), cache, rows, lens.cuda(), NOPE, PE)
    for r, n in enumerate(lens.tolist()):
        if n <= 0:
            assert not O[r].any() and (lse[r] == -np.inf).all()
            continue
        t = np.arange(n)
        k = values[table[r // chunk].numpy()[t // page].astype(np.int64) * page + t % page]
        want, wantL, tol, tolL = L.attention(f64(q[r]), k, np.ones(n, bool), D ** -0.5)
        assert (np.abs(f64(O[r]) - want) <= tol).all() and (np.abs(f64(lse[r]) - wantL) <= tolL).all(), (r, n)


def test_e4m3_rows_beyond_four_gigabytes():
    page, nh = 64, 64
    pages = 8 * 2**20 // page
    cache = ir.kv_latent_empty(pages, page, NOPE, PE, E4M3)
    assert cache.numel() > 2**32
    x = torch.randn(256, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    at = torch.arange((pages - 4) * page, pages * page, dtype=torch.int32, device="cuda")
    ir.kv_latent_write(cache, x, at, NOPE, PE)
    values = f64(ir.kv_latent_read(cache, at, NOPE, PE))
    q = torch.randn(1, nh, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    table = torch.tensor([[pages - 1, pages - 4, pages - 2]], dtype=torch.int32, device="cuda")
    got = [ir.latent_attn_decode(q.cuda(), cache, table, torch.tensor([150], dtype=torch.int32, device="cuda"), NOPE, PE)]
    order = np.concatenate([np.arange(192, 256), np.arange(0, 64), np.arange(128, 150)])
    idx = torch.from_numpy(order.astype(np.int32)).cuda()[None] + (pages - 4) * page
    got.append(ir.latent_attn_sparse(q.cuda(), cache, idx.contiguous(), NOPE, PE))
    want, wantL, tol, tolL = L.attention(f64(q[0]), values[order], np.ones(150, bool), D ** -0.5)
    for O, lse in got:
        assert (np.abs(f64(O[0]) - want) <= tol).all() and (np.abs(f64(lse[0]) - wantL) <= tolL).all()


def test_calls_from_several_host_threads():
    """Each with its stream: first calls at once, then many."""
    batches = [_batch(rows=3 + k, pages=4 + 3 * k, nh=[64, 128, 5, 40][k], fmt=[BF16, E4M3][k % 2], seed=k)
               for k in range(4)]
    want = [ir.latent_attn_decode(*b, NOPE, PE) for b in batches]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(4), []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            start.wait(timeout=60)
            for _ in range(25):
                O, lse = ir.latent_attn_decode(*batches[k], NOPE, PE, stream=stream)
                slots = torch.arange(8, dtype=torch.int32, device="cuda")
                stream.synchronize()
                assert torch.equal(O, want[k][0]) and torch.equal(lse, want[k][1])
                torch.cuda.current_stream().synchronize()
                ir.kv_latent_read(batches[k][1], slots, NOPE, PE, stream=stream)
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
