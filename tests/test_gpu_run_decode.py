"""The operators in the order of a decoder layer (``run_decode``): prompt written,
selected tokens attended to, decoding steps, against the fp64 oracles composed
alike. Needs a GB300."""

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


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _check(Y, q, values, slots_of, M, positions, nope, pe):
    """Attention's tolerance goes through the rotation (at most sqrt 2 of a pair's
    larger) and the mix (a row's absolute sum); the postmix adds its own."""
    Q, M = f64(q), f64(M)
    O, tol = np.zeros_like(Q), 0.0
    for r in range(len(Q)):
        s = np.asarray(slots_of(r), dtype=np.int64)
        O[r], _, tolO, _ = L.attention(Q[r], values[np.maximum(s, 0)], s >= 0, (nope + pe) ** -0.5)
        tol = max(tol, tolO.max())
    want = oracle.postmix_fwd(O, M, positions, nope, pe, 10000.0)
    allowed = 2.0 ** 0.5 * np.abs(M).sum(1).max() * tol + 8e-3 * np.abs(want).max()
    assert np.abs(f64(Y) - want).max() <= allowed


@pytest.mark.parametrize("fmt", [ir.KV_LATENT_BF16, ir.KV_LATENT_E4M3])
@pytest.mark.parametrize("rows,nh,page", [(3, 8, 16), (1, 64, 64), (5, 5, 7)])
def test_prompt_selection_and_steps(fmt, rows, nh, page):
    nope, pe, chunk, topk = 448, 64, 4, 33
    d, dev = nope + pe, "cuda"
    server = run_decode.Server(rows, 150, nh, nope, pe, page, fmt, seed=rows)
    lens = torch.tensor([100, 37, 1, 64, 140][:rows], dtype=torch.int32, device=dev)
    server.prompt(W.normal_bf16((int(lens.sum()), d), 1, device=dev), lens)
    every = torch.arange(rows * server.capacity, dtype=torch.int32, device=dev)
    begin = np.arange(rows) * server.capacity

    held = [slice(begin[r], begin[r] + int(lens[r])) for r in range(rows)]
    values = np.zeros((len(every), d))
    now = f64(ir.kv_latent_read(server.cache, every, nope, pe))
    for h in held:
        values[h] = now[h]
    rng = np.random.default_rng(rows)
    idx = rng.integers(-1, np.repeat(lens.cpu().numpy(), chunk)[:, None], (rows * chunk, topk)).astype(np.int32)
    q = W.normal_bf16((rows * chunk, nh, d), 2, device=dev)
    at = torch.arange(rows * chunk, dtype=torch.int32, device=dev)
    Y = server.selected(q, torch.from_numpy(idx).to(dev), at)
    _check(Y, q, values, lambda r: np.where(idx[r] < 0, -1, idx[r] + begin[r // chunk]), server.M,
           np.arange(rows * chunk), nope, pe)

    for step in range(3):
        x, q = W.normal_bf16((rows, d), 10 + step, device=dev), W.normal_bf16((rows, nh, d), 20 + step, device=dev)
        Y = server.step(x, q)
        n = lens.cpu().numpy().astype(np.int64) + step + 1
        assert server.lens.cpu().tolist() == n.tolist()
        now = f64(ir.kv_latent_read(server.cache, every, nope, pe))
        _check(Y, q, now, lambda r: begin[r] + np.arange(n[r]), server.M, n - 1, nope, pe)


@pytest.mark.parametrize("extra", [[], ["--graph"], ["--fmt", "bf16", "--nh", "16", "--page", "16"]])
def test_command(extra, capsys):
    assert run_decode.main(["--rows", "3", "--prompt", "300", "--steps", "4", "--topk", "64"] + extra) == 0
    assert "finite: True" in capsys.readouterr().out
