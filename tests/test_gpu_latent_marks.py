"""Long rows of the latent attention, split over thread blocks and joined, with
values that show the loss of a tile or of a token (``latent_marks``; what they show
is tested in ``test_latent_oracle_loss.py``). Needs a GB300."""

import numpy as np
import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built, f64
from latent_marks import marked
from oracle import latent_oracle as L

pytestmark = pytest.mark.gpu

BF16, E4M3 = ir.KV_LATENT_BF16, ir.KV_LATENT_E4M3
NOPE, PE, D = 448, 64, 512


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _written(values, slots, num_slots, page, fmt):
    cache = ir.kv_latent_empty(num_slots // page, page, NOPE, PE, fmt)
    cache.view(torch.uint8).fill_(0xFF)  # NaN in what is not attended to
    ir.kv_latent_write(cache, torch.from_numpy(values).to(torch.bfloat16).cuda(), torch.from_numpy(slots).cuda(), NOPE, PE)
    back = f64(ir.kv_latent_read(cache, torch.from_numpy(slots).cuda(), NOPE, PE))
    assert np.array_equal(back, values)  # 0 and 1 have codes
    return cache


def _queries(rows, nh, size, seed):
    return (size * torch.randn(rows, nh, D, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def _check(q, values_of, O, lse):
    for r in range(len(q)):
        v = values_of(r)
        want, wantL, tol, tolL = L.attention(f64(q[r]), v, np.ones(len(v), bool), D ** -0.5)
        off = np.abs(f64(O[r]) - want) - tol
        assert (off <= 0).all(), f"row {r} of {len(v)}: channels {np.unique(np.nonzero(off > 0)[1])[:20]}"
        if len(v):
            assert (np.abs(f64(lse[r]) - wantL) <= tolL).all()


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("per", ["tile", "token"])
@pytest.mark.parametrize("size", [0.0, 0.5])
@pytest.mark.parametrize("lens,nh,page", [
    ([20011], 8, 64), ([65536], 2, 64), ([9000, 17, 4096, 0, 12345, 64, 1], 128, 16), ([700] * 40, 3, 7),
    ([3001 + 64 * r for r in range(33)], 5, 64),
])
def test_every_tile_of_a_long_row_counts(fmt, per, size, lens, nh, page):
    if per == "token" and max(lens) > 20011:
        pytest.skip("one of 65536 tokens is within the tolerance")
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    order = np.random.default_rng(len(lens)).permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(need)), -1, np.int32)
    values, slots, at = [], [], 0
    for r, n in enumerate(lens):
        table[r, :need[r]] = order[at:at + need[r]]
        at += need[r]
        t = np.arange(n)
        values.append(marked(n, D, per))
        slots.append(table[r, t // page].astype(np.int64) * page + t % page)
    cache = _written(np.concatenate(values), np.concatenate(slots).astype(np.int32), pages * page, page, fmt)
    q = _queries(len(lens), nh, size, nh)
    O, lse = ir.latent_attn_decode(q.cuda(), cache, torch.from_numpy(table).cuda(),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), NOPE, PE)
    _check(q, lambda r: values[r], O, lse)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("rows,topk", [(2, 9000), (70, 2048)])
def test_every_selected_row_counts(fmt, rows, topk):
    n = 20032
    cache = _written(marked(n, D, "token"), np.arange(n, dtype=np.int32), n, 64, fmt)
    rng = np.random.default_rng(topk)
    idx = np.stack([rng.permutation(n)[:topk] for _ in range(rows)]).astype(np.int32)
    q = _queries(rows, 6, 0.5, topk)
    O, lse = ir.latent_attn_sparse(q.cuda(), cache, torch.from_numpy(idx).cuda(), NOPE, PE)
    values = marked(n, D, "token")
    _check(q, lambda r: values[idx[r]], O, lse)
