"""Random shapes of the latent attention: formats, channel splits, heads, pages and
ragged lengths with empty rows among them, each three times with the same bits,
against fp64 torch on the GPU with the oracle's tolerances. Half of the cases have
values that show the loss of a few tokens. (Races between a row's end and the next
row's beginning showed in such shapes alone.) Needs a GB300."""

import random

import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu

BF16, E4M3 = ir.KV_LATENT_BF16, ir.KV_LATENT_E4M3


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _reference(q, k, scale):
    """``oracle.latent_oracle.attention`` of one row, in fp64 on the GPU."""
    n, d = k.shape
    s = scale * (q @ k.T)
    m = s.amax(1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(1, keepdim=True)
    p = p / total
    ds = (abs(scale) * (d + 2) * 2.0 ** -24) * (q.abs() @ k.abs().T).amax(1)
    O = p @ k
    tol = (p @ k.abs()) * (2.0 ** -8 + 2 * ds[:, None] + 2.0 ** -21 + n * 2.0 ** -23) + O.abs() * 2.0 ** -8
    lse = (m + torch.log(total))[:, 0]
    return O, lse, tol, ds + 2.0 ** -21 + n * 2.0 ** -24 + (lse.abs() + m[:, 0].abs()) * 2.0 ** -22


def _shape(rng):
    fmt = rng.choice([BF16, E4M3])
    if rng.random() < 0.4:
        nope, pe = 448, 64
    elif fmt == E4M3:
        nope = 16 * rng.randint(1, 32)
        pe = 8 * rng.randint(0, (512 - nope) // 8)
    else:
        d = 8 * rng.randint(1, 64)
        nope = rng.randint(0, d)
        pe = d - nope
    rows = rng.choice([1, 1, 2, 3, 7, 20, 60, 200, 400])
    longest = int(10 ** rng.uniform(0, 4.5 if rows < 4 else 3.7 if rows < 25 else 2.7))
    lens = [rng.choice([0, 1, longest, rng.randint(0, longest)]) for _ in range(rows)]
    return fmt, nope, pe, rng.choice([1, 2, 3, 5, 8, 16, 17, 40, 64, 64, 64, 65, 100, 128]), \
        rng.choice([1, 3, 8, 16, 64, 64, 100, 256]), lens


@pytest.mark.parametrize("seed", range(60))
def test_random_shape(seed):
    rng = random.Random(seed)
    fmt, nope, pe, nh, page, lens = _shape(rng)
    d, rows = nope + pe, len(lens)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.full((rows, max(need + [1])), -1, dtype=torch.int32, device="cuda")
    slots, at = [], 0
    for r, k in enumerate(need):
        table[r, :k] = order[at:at + k]
        at += k
        t = torch.arange(lens[r], device="cuda")
        slots.append(table[r].long()[t // page] * page + t % page)
    held = torch.cat(slots)
    x = torch.randn(len(held), d, generator=gen, device="cuda")
    if rng.random() < 0.5:  # one channel of each token, other tokens' nearly zero there
        x *= rng.choice([0.0, 2.0 ** -9])
        ch = torch.randint(0, d, (len(held),), generator=gen, device="cuda")
        x[torch.arange(len(held), device="cuda"), ch] = 1 + torch.rand(len(held), generator=gen, device="cuda")
    cache = ir.kv_latent_empty(pages, page, nope, pe, fmt)
    cache.view(torch.uint8).fill_(0xFF)  # NaN in what is not attended to
    ir.kv_latent_write(cache, x.to(torch.bfloat16), held.int(), nope, pe)
    values = ir.kv_latent_read(cache, torch.arange(pages * page, dtype=torch.int32, device="cuda"), nope, pe).double()
    q = (torch.randn(rows, nh, d, generator=gen, device="cuda") * rng.choice([0.0, 0.3, 1.0, 4.0])).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    (O, lse), *again = [ir.latent_attn_decode(q, cache, table, n, nope, pe) for _ in range(3)]
    for O1, lse1 in again:
        assert torch.equal(O1, O) and torch.equal(lse1, lse)
    for r in range(rows):
        if lens[r] == 0:
            assert not O[r].any() and (lse[r] == -float("inf")).all()
            continue
        want, wantL, tol, tolL = _reference(q[r].double(), values[slots[r]], d ** -0.5)
        assert ((O[r].double() - want).abs() <= tol).all(), r
        assert ((lse[r].double() - wantL).abs() <= tolL).all(), r
