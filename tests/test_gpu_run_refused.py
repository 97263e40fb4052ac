"""``run_decode.PooledServer`` when the pool has no page: which sequences took a step, what
the others' rows are worth, and their step asked for again. Needs a GB300."""

import numpy as np
import pytest
import torch

import oracle
import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built, f64
from oracle import latent_oracle as L
from oracle import rope_oracle as R
from partial_inverse_rope_gb300 import binding
from partial_inverse_rope_gb300 import inputs as W
from partial_inverse_rope_gb300 import run_decode

pytestmark = pytest.mark.gpu

ROWS, NH, NOPE, PE, PAGE = 4, 3, 64, 32, 4
D = NOPE + PE


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _turned(x, server, positions):
    """bf16 vectors at these positions, as float64: the call's own rounding, within its tolerance."""
    got = f64(ir.rope_apply(x, server.freqs, torch.tensor(positions, dtype=torch.int32, device="cuda")))
    want, size = R.rope(f64(x).reshape(len(x), -1, D), server.freqs.numpy(), np.array(positions), NOPE, 1.0, False, False)
    assert (np.abs(got.reshape(want.shape) - want) <= R.tolerance(want, size, "bf16")).all()
    return got


@pytest.mark.parametrize("graph", [False, True])
def test_refused_sequences_are_named_and_ask_again(graph):
    """Four sequences of 3, 4, 8 and 2 tokens, pages of 4, a pool of 5: two of them
    stand before a new page, which the pool does not have."""
    server = run_decode.PooledServer(ROWS, 32, 5, NH, NOPE, PE, PAGE, ir.KV_LATENT_BF16)
    x, q = W.normal_bf16((ROWS, D), 1, device="cuda"), W.normal_bf16((ROWS, NH, D), 2, device="cuda")
    if graph:
        start = [t.clone() for t in (server.state, server.table, server.queue)]
        server.step(x, q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y = server.step(x, q)
        for t, was in zip((server.state, server.table, server.queue), start):
            t.copy_(was)
    lens = [3, 4, 8, 2]
    first = W.normal_bf16((sum(lens), D), 3, device="cuda")
    assert server.prompt(first, torch.tensor(lens, dtype=torch.int32, device="cuda")).tolist() == lens
    X = _turned(first, server, [t for n in lens for t in range(n)])
    held = [X[sum(lens[:i]):sum(lens[:i + 1])] for i in range(ROWS)]
    M = f64(server.M)

    def one(seed, want):
        nonlocal Y
        x.copy_(W.normal_bf16((ROWS, D), seed, device="cuda"))
        q.copy_(W.normal_bf16((ROWS, NH, D), seed + 1, device="cuda"))
        if graph:
            g.replay()
        else:
            Y = server.step(x, q)
        assert server.granted.tolist() == want
        where = [len(h) for h in held]  # where each sequence's next token stands, taken or not
        new, Q = _turned(x, server, where), _turned(q, server, where)
        for i in range(ROWS):
            if not want[i]:
                continue
            held[i] = np.concatenate([held[i], new[i:i + 1]])
            O, _, tol, _ = L.attention(Q[i], held[i], np.ones(len(held[i]), bool), D ** -0.5)
            answer = oracle.postmix_fwd(O[None], M, np.array([where[i]]), NOPE, PE, 10000.0)[0]
            allowed = 2.0 ** 0.5 * np.abs(M).sum(1).max() * tol.max() + 8e-3 * np.abs(answer).max()
            assert np.abs(f64(Y[i]) - answer).max() <= allowed
        assert server.lens.tolist() == [len(h) for h in held]

    if not graph:
        Y = None
    one(10, [1, 0, 0, 1])      # no page is left: 1 + 1 + 2 + 1
    one(20, [0, 0, 0, 1])
    server.prompt(x[:0], torch.tensor([0, 0, -1, 0], dtype=torch.int32, device="cuda"))
    held[2] = held[2][:0]      # its two pages come back
    one(30, [1, 1, 0, 0])      # (the queue is first come, first served: rows 2 and 3 get none)
    one(40, [1, 1, 0, 0])


def test_no_sequence_took_a_step_before_the_first():
    server = run_decode.PooledServer(ROWS, 32, 5, NH, NOPE, PE, PAGE, ir.KV_LATENT_BF16)
    assert server.granted.tolist() == [0] * ROWS


def test_a_step_into_given_tensors(monkeypatch):
    """Through the compiled call and without it: the same numbers, in the caller's tensors."""
    if binding._calls is None:
        pytest.skip("the compiled calls were not built")
    first = ir.kv_pages_empty(6, 5, 9)
    new = torch.tensor([3, 0, 70, -1, 16, 1], dtype=torch.int32, device="cuda")
    sizes, got = (100, 100, 100, 7, 6), []
    for way in (binding._calls, None):
        monkeypatch.setattr(binding, "_calls", way)
        state, table, queue = [t.clone() for t in first]
        out = [torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in sizes]
        back = ir.kv_pages_advance(state, table, queue, new, 16, 100, out=out)
        assert type(back) is tuple and all(a is b for a, b in zip(back, out, strict=True))
        got.append([t.tolist() for t in (*out, state, table, queue)])
        for k in range(5):
            wrong = [*out[:k], torch.zeros(sizes[k] + 1, dtype=torch.int32, device="cuda"), *out[k + 1:]]
            with pytest.raises(ValueError, match="must be"):
                ir.kv_pages_advance(state, table, queue, new, 16, 100, out=wrong)
        with pytest.raises(ValueError):
            ir.kv_pages_advance(state, table, queue, new, 16, 100, out=out[:4])
        with pytest.raises(ir.InvropeError, match="INVALID_ARG"):  # one tensor twice
            ir.kv_pages_advance(state, table, queue, new, 16, 100, out=[out[0], out[0], *out[2:]])
        assert state.tolist() == got[-1][5]
    assert got[0] == got[1]
