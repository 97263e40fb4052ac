"""Scores of -inf in the attention over the latent cache: they have no weight
beside others, and where there are no others the output is 0 / 0, not the zeros
of a row with nothing to attend to. Needs a GB300."""

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


def _cache(n, fmt, seed, change=None):
    x = torch.randn(n, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    if change is not None:
        change(x)
    cache = ir.kv_latent_empty(n, 1, NOPE, PE, fmt)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    ir.kv_latent_write(cache, x.cuda(), slots, NOPE, PE)
    return cache, f64(ir.kv_latent_read(cache, slots, NOPE, PE))


def _q(rows, nh, seed):
    return torch.randn(rows, nh, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("n", [1, 64, 70, 3000])  # one tile to a row split over many blocks
def test_an_infinite_query_of_scores_all_below_shows(fmt, n):
    cache, values = _cache(n, fmt, n, lambda x: x[:, 500].fill_(1.0))
    q = _q(2, 5, n)
    q[:, 3, 500] = float("-inf")
    idx = torch.arange(n, dtype=torch.int32).repeat(2, 1)
    idx[1] = -1  # and nothing to attend to
    O, lse = ir.latent_attn_sparse(q.cuda(), cache, idx.cuda(), NOPE, PE)
    assert torch.isnan(O[0, 3]).all() and lse[0, 3] == -np.inf
    assert not O[1].any() and (lse[1] == -np.inf).all()
    keep = [0, 1, 2, 4]
    want, wantL, tol, tolL = L.attention(f64(q[0, keep]), values, np.ones(n, bool), D ** -0.5)
    assert (np.abs(f64(O[0, keep]) - want) <= tol).all() and (np.abs(f64(lse[0, keep]) - wantL) <= tolL).all()


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("n,low", [(70, slice(0, 64)), (70, slice(64, 70)), (70, slice(3, 69)), (3000, slice(0, 900)),
                                   (3000, slice(700, 3000)), (3000, slice(0, 2999))])
def test_scores_of_minus_infinity_beside_others_have_no_weight(fmt, n, low):
    """They come of products beyond fp32's range; the tokens' values are finite."""
    def change(x):
        x[:, 500] = 0
        x[low, 500] = -(2.0 ** 90)
    cache, values = _cache(n, fmt, n, change)
    q = _q(1, 4, n)
    q[0, :, 500] = torch.tensor([2.0 ** 90, 0.0, 2.0 ** 90, 0.0])
    heads = [0, 2]
    O, lse = ir.latent_attn_sparse(q.cuda(), cache, torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous(),
                                   NOPE, PE)
    valid = np.ones(n, bool)
    valid[low] = False
    want, wantL, tol, tolL = L.attention(f64(q[0, heads]), values, valid, D ** -0.5)
    assert (np.abs(f64(O[0, heads]) - want) <= tol).all() and (np.abs(f64(lse[0, heads]) - wantL) <= tolL).all()
