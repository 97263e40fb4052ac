"""Steps of a pool with prompts, in two launches: captured and replayed, in place or not, and
with exactly the pages, tokens and places that there are. Needs a GB300."""

import numpy as np
import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built
from oracle import pages_oracle as P

pytestmark = pytest.mark.gpu

NAMES = ("slots", "positions", "rows", "starts", "granted")


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("b,room", [(40, 4000), (2500, 3000), (5000, 0)])
def test_captured_steps_of_two_launches(b, room, in_place):
    """More than 2048 tokens and sequences: the state is written by the second launch. A graph
    of two steps, replayed, beside steps of another pool on another stream."""
    rng = np.random.default_rng(b)
    page, width = 16, 30
    pages = 20 * b
    state, table, queue = ir.kv_pages_empty(b, width, pages)
    after = state if in_place else torch.empty_like(state)
    new = torch.zeros(b, dtype=torch.int32, device="cuda")
    sizes = (room, room, room, b + 1, b)
    outs = [[torch.empty(n, dtype=torch.int32, device="cuda") for n in sizes] for _ in range(2)]
    other, asked = ir.kv_pages_empty(3, 500, 1500), torch.full((3,), 1000, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ir.kv_pages_advance(state, table, queue, new, page, room, state_out=after, out=outs[0])
        ir.kv_pages_advance(after, table, queue, new, page, room, state_out=state, out=outs[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s, t, q = [x.cpu().numpy() for x in (state, table, queue)]
    for k in range(6):
        n = np.where(rng.random(b) < 0.1, -1, rng.integers(0, max(2, 3 * room // (2 * b)), b)).astype(np.int32)
        n[rng.integers(0, b, 3)] = rng.integers(1, 400, 3)
        new.copy_(torch.from_numpy(n))
        graph.replay()
        ir.kv_pages_advance(*other, asked, 64, 3000, stream=side)
        torch.cuda.synchronize()
        for out in outs:
            want = P.advance(s, t, q, n, page, room)
            s, t, q = want["state"], want["table"], want["queue"]
            for name, got in zip(NAMES, out):
                assert np.array_equal(got.cpu().numpy(), want[name]), (k, name)
        for name, got in zip(("state", "table", "queue"), (state, table, queue)):
            assert np.array_equal(got.cpu().numpy(), want[name]), (k, name)
    assert other[0].tolist()[:3] == [6000] * 3 and int(other[0][-1]) == 1500 - 3 * -(-6000 // 64)


@pytest.mark.parametrize("more", [0, 3000])
@pytest.mark.parametrize("free,want", [(3, [8, 4]), (2, [8, 0]), (1, [0, 0]), (0, [0, 0])])
def test_as_many_pages_as_there_are(free, want, more):
    """Sequences of 4 and 0 tokens ask for 8 and 4, pages of 4: two pages and one. (With one
    page the first gets nothing, and the second neither: its page would be the third asked for.)"""
    table = np.full((2, 4), -1, np.int32)
    table[0, 0] = free
    queue = np.arange(free + 1, dtype=np.int32)
    state = np.array([4, 0, 0, free], np.int32)
    gpu = [torch.from_numpy(x).cuda() for x in (state, table, queue, np.array([8, 4], np.int32))]
    got = ir.kv_pages_advance(*gpu, 4, 50 + more)
    assert got[4].tolist() == want and gpu[0].tolist()[:2] == [4 + want[0], want[1]]
    oracle = P.advance(state, table, queue, [8, 4], 4, 50 + more)
    for name, x in zip((*NAMES, "state", "table", "queue"), (*got, *gpu)):
        assert np.array_equal(x.cpu().numpy(), oracle[name]), name
