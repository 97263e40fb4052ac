"""Writing the latent cache and reading it back, against the fp64 oracle: codes,
scale bytes and values have to be equal, bit for bit. Needs a GB300."""

import numpy as np
import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built, f64
from oracle import latent_oracle as L

pytestmark = pytest.mark.gpu

BF16, E4M3 = ir.KV_LATENT_BF16, ir.KV_LATENT_E4M3


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _vectors(n, d, seed):
    """Normal vectors whose groups differ in size by many powers of two."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-30, 30, (n, -(-d // 8)), generator=g).float()).repeat_interleave(8, 1)[:, :d]
    return (torch.randn(n, d, generator=g) * size).to(torch.bfloat16)


def _cache(pages, page, nope, pe, fmt, fill=0xA5):
    c = ir.kv_latent_empty(pages, page, nope, pe, fmt)
    c.view(torch.uint8).fill_(fill)
    return c


SPLITS = [(448, 64), (480, 32), (96, 32), (64, 64), (48, 16), (16, 0), (16, 8), (512, 0), (112, 8), (16, 496)]


@pytest.mark.parametrize("nope,pe", SPLITS)
@pytest.mark.parametrize("n", [1, 3, 130])
def test_write_stores_the_codes_and_scales_of_the_definition(nope, pe, n):
    d, page = nope + pe, 16
    x = _vectors(n, d, 10 * n + nope)
    cache = _cache(12, page, nope, pe, E4M3)
    slots = torch.randperm(12 * page, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    before = cache.clone()
    assert ir.kv_latent_write(cache, x.cuda(), slots.cuda(), nope, pe) is cache
    got = cache.view(12 * page, -1).cpu().numpy()
    codes, scales = L.quantise(f64(x), nope)
    rows = got[slots.numpy()]
    assert np.array_equal(rows[:, :nope], codes)
    assert np.array_equal(rows[:, nope:nope + 2 * pe], x[:, nope:].contiguous().view(torch.uint8).numpy())
    groups = scales.shape[1]
    assert np.array_equal(rows[:, nope + 2 * pe:nope + 2 * pe + groups], scales)
    assert (rows[:, nope + 2 * pe + groups:] == 0xA5).all()
    rest = np.setdiff1d(np.arange(12 * page), slots.numpy())
    assert np.array_equal(got[rest], before.view(12 * page, -1).cpu().numpy()[rest])
    back = ir.kv_latent_read(cache, slots.cuda(), nope, pe)
    assert np.array_equal(f64(back[:, :nope]), L.dequantise(codes, scales))  # exact in bf16
    assert torch.equal(back[:, nope:].cpu(), x[:, nope:])


@pytest.mark.parametrize("nope,pe", SPLITS + [(0, 8), (6, 2), (8, 0), (450, 62)])
def test_bf16_rows_keep_their_bits(nope, pe):
    d = nope + pe
    x = torch.randint(-32768, 32767, (77, d), generator=torch.Generator().manual_seed(d)).to(torch.int16)
    x = x.view(torch.bfloat16)  # every kind of value, NaN and infinities among them
    cache = _cache(5, 48, nope, pe, BF16)
    slots = torch.randperm(240, generator=torch.Generator().manual_seed(1))[:77].to(torch.int32).cuda()
    ir.kv_latent_write(cache, x.cuda(), slots, nope, pe)
    back = ir.kv_latent_read(cache, slots, nope, pe)
    assert torch.equal(back.cpu().view(torch.int16), x.view(torch.int16))
    assert torch.equal(cache.view(240, d)[slots.long()].cpu().view(torch.int16), x.view(torch.int16))


def test_values_at_the_edges_of_the_formats():
    nope = 64
    tiny, big = 2.0**-133, float(torch.finfo(torch.bfloat16).max)
    groups = [
        [0.0], [-0.0, 0.0], [tiny], [tiny, -2.0**-126], [448.0], [450.0, 1.0], [1.75, 0.001], [1.7578125],
        [big, -big, 1.0], [1.75 * 2.0**127, 2.0**118], [2.0**-111 * 1.75, 2.0**-120], [2.0**-112, 2.0**-130],
        [448.0, 17.0, 19.0, 18.0, 2.0**-9, 1.5 * 2.0**-9, 2.0**-10, 1.0625, 1.1875],
        [float("inf"), 1.0], [1.0, float("-inf")], [float("nan")], [3.0, 5.0, -7.0],
    ]
    x = torch.zeros(len(groups), nope + 8)
    for i, g in enumerate(groups):
        x[i, :len(g)] = torch.tensor(g)
    x = x.to(torch.bfloat16)
    cache = _cache(2, 16, nope, 8, E4M3, fill=0)
    slots = torch.arange(len(groups), dtype=torch.int32).cuda()
    ir.kv_latent_write(cache, x.cuda(), slots, nope, 8)
    codes, scales = L.quantise(f64(x), nope)
    rows = cache.view(32, -1)[:len(groups)].cpu().numpy()
    assert np.array_equal(rows[:, 80], scales[:, 0])
    finite = scales[:, 0] != 255
    assert finite.sum() == len(groups) - 3
    assert np.array_equal(rows[finite, :nope], codes[finite])
    back = f64(ir.kv_latent_read(cache, slots, nope, 8))
    want = L.dequantise(codes, scales)
    assert np.array_equal(back[:, :nope], want, equal_nan=True)
    assert np.isnan(back[~finite, :nope]).all() and not back[:, nope:].any()


def test_every_code_and_scale_reads_as_its_value():
    """All e4m3 codes but the two NaN ones (which the writer never stores) under
    every scale byte the writer stores, and the NaN byte."""
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    codes = np.concatenate([codes, codes[:2]]).reshape(1, 256)
    scale = np.array(list(range(7, 247)) + [255], np.uint8)
    rows = np.zeros((len(scale), 272), np.uint8)
    rows[:, :256] = codes
    rows[:, 256:260] = scale[:, None]
    cache = torch.from_numpy(rows).view(len(scale), 1, 272).cuda()
    back = f64(ir.kv_latent_read(cache, torch.arange(len(scale), dtype=torch.int32).cuda(), 256, 0))
    want = L.dequantise(np.repeat(codes, len(scale), 0), np.repeat(scale[:, None], 4, 1))
    assert np.array_equal(back, want, equal_nan=True)
    top = back[scale == 246]
    assert np.isfinite(top).all()


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_slots_out_of_range_store_and_read_nothing(fmt):
    nope, pe = 96, 32
    x = _vectors(6, 128, 5).cuda()
    cache = _cache(3, 8, nope, pe, fmt)
    before = cache.clone()
    bad = torch.tensor([-1, 24, -2**31, 2**31 - 1, 25, -24], dtype=torch.int32).cuda()
    ir.kv_latent_write(cache, x, bad, nope, pe)
    assert torch.equal(cache.view(torch.uint8), before.view(torch.uint8))
    assert not ir.kv_latent_read(cache, bad, nope, pe).any()
    some = torch.tensor([-1, 23, 24, 0, 5, -7], dtype=torch.int32).cuda()
    ir.kv_latent_write(cache, x, some, nope, pe)
    back = ir.kv_latent_read(cache, some, nope, pe)
    assert back[[1, 3, 4]].any(1).all() and not back[[0, 2, 5]].any()


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_no_tokens(fmt):
    cache = _cache(1, 4, 48, 16, fmt)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    ir.kv_latent_write(cache, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), none, 48, 16)
    assert ir.kv_latent_read(cache, none, 48, 16).shape == (0, 64)


@pytest.mark.parametrize("fmt,slots", [(BF16, 5 * 2**20), (E4M3, 8 * 2**20)])
def test_rows_beyond_four_gigabytes(fmt, slots):
    nope, pe = 448, 64
    cache = ir.kv_latent_empty(slots // 64, 64, nope, pe, fmt)
    assert cache.numel() * cache.element_size() > 2**32
    x = _vectors(64, 512, 9)
    at = torch.cat([torch.arange(32), torch.arange(slots - 32, slots)]).to(torch.int32)
    ir.kv_latent_write(cache, x.cuda(), at.cuda(), nope, pe)
    back = f64(ir.kv_latent_read(cache, at.cuda(), nope, pe))
    want = f64(x)
    if fmt == E4M3:
        want[:, :nope] = L.dequantise(*L.quantise(want, nope))
    assert np.array_equal(back, want)


def test_on_a_stream_of_its_own_and_in_a_graph():
    nope, pe = 448, 64
    x = _vectors(300, 512, 2).cuda()
    slots = torch.randperm(512)[:300].to(torch.int32).cuda()
    ref = ir.kv_latent_read(ir.kv_latent_write(_cache(8, 64, nope, pe, E4M3), x, slots, nope, pe), slots, nope, pe)
    s = torch.cuda.Stream()
    cache = _cache(8, 64, nope, pe, E4M3)
    s.wait_stream(torch.cuda.current_stream())
    ir.kv_latent_write(cache, x, slots, nope, pe, stream=s)
    out = ir.kv_latent_read(cache, slots, nope, pe, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(ref)
    with torch.cuda.graph(graph):
        ir.kv_latent_write(cache, x, slots, nope, pe)
        ir.kv_latent_read(cache, slots, nope, pe, out=out)
    for k in range(2):
        x.copy_(_vectors(300, 512, 50 + k))
        cache.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        codes, scales = L.quantise(f64(x), nope)
        assert np.array_equal(f64(out[:, :nope]), L.dequantise(codes, scales))
