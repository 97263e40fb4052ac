"""A server (``run_decode``) whose sequences are full: their next tokens take the
last one's place, and fall into no other sequence's pages. Needs a GB300."""

import numpy as np
import pytest
import torch

import oracle
import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built, f64
from oracle import latent_oracle as L
from partial_inverse_rope_gb300 import inputs as W
from partial_inverse_rope_gb300 import run_decode

pytestmark = pytest.mark.gpu

NOPE, PE, NH, D = 48, 16, 4, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_full_sequences_keep_to_their_own_pages(graph):
    server = run_decode.Server(3, 32, NH, NOPE, PE, 16, ir.KV_LATENT_BF16)
    lens = torch.tensor([32, 30, 31], dtype=torch.int32, device="cuda")
    server.prompt(W.normal_bf16((int(lens.sum()), D), 1, device="cuda"), lens)
    every = torch.arange(96, dtype=torch.int32, device="cuda")
    held = ir.kv_latent_read(server.cache, every, NOPE, PE).cpu()
    x, q = W.normal_bf16((3, D), 2, device="cuda"), W.normal_bf16((3, NH, D), 3, device="cuda")
    step, Y = (lambda: server.step(x, q)), None
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y = server.step(x, q)
        step = g.replay
    for k in range(4):
        x.copy_(W.normal_bf16((3, D), 10 + k, device="cuda"))
        for r in range(3):
            held[32 * r + min(int(lens[r]) + k, 31)] = x[r].cpu()
        out = step()
        out = Y if graph else out
        now = ir.kv_latent_read(server.cache, every, NOPE, PE).cpu()
        n = np.minimum(lens.cpu().numpy() + k + 1, 32)
        for r in range(3):
            assert torch.equal(now[32 * r:32 * r + n[r]], held[32 * r:32 * r + n[r]]), (k, r)
        # a token of the row next to it would show here too
        O, tol = np.zeros((3, NH, D)), 0.0
        for r in range(3):
            O[r], _, tolO, _ = L.attention(f64(q[r]), f64(held[32 * r:32 * r + n[r]]), np.ones(n[r], bool), D ** -0.5)
            tol = max(tol, tolO.max())
        M = f64(server.M)
        want = oracle.postmix_fwd(O, M, lens.cpu().numpy().astype(np.int64) + k, NOPE, PE, 10000.0)
        # through the rotation (at most sqrt 2 of a pair's larger) and the mix, and the postmix's own
        allowed = 2.0 ** 0.5 * np.abs(M).sum(1).max() * tol + 8e-3 * np.abs(want).max()
        assert np.abs(f64(out) - want).max() <= allowed


def test_a_prompt_longer_than_a_sequence_is_refused():
    server = run_decode.Server(2, 32, NH, NOPE, PE, 16, ir.KV_LATENT_BF16)
    lens = torch.tensor([3, 33], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="33 tokens"):
        server.prompt(W.normal_bf16((36, D), 1, device="cuda"), lens)


@pytest.mark.parametrize("extra", [[], ["--graph"]])
def test_command_without_steps(extra, capsys):
    assert run_decode.main(["--rows", "2", "--prompt", "100", "--steps", "0", "--topk", "16"] + extra) == 0
    assert "finite: True" in capsys.readouterr().out
