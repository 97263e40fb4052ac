"""Attention over the latent cache, paged and by index table, against the fp64
oracle, whose element-wise tolerances count the kernel's roundings (see
``oracle.latent_oracle.attention``). Needs a GB300."""

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


def _pool(pages, page, nope, pe, fmt, seed):
    """A written cache and its values, float64 [slots, d]."""
    d, n = nope + pe, pages * page
    x = torch.randn(n, d, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    cache = ir.kv_latent_empty(pages, page, nope, pe, fmt)
    cache.view(torch.uint8).fill_(0xFF)  # padding
    ir.kv_latent_write(cache, x, slots, nope, pe)
    return cache, f64(ir.kv_latent_read(cache, slots, nope, pe))


def _q(rows, nh, d, seed, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, nh, d, generator=g, device="cuda") * size).to(torch.bfloat16)


def _check(q, values, slots_of, scale, O, lse):
    """Every row against the oracle; slots_of(r) gives its slots, -1 where left out."""
    Q, O, lse = f64(q), f64(O), f64(lse)
    for r in range(len(Q)):
        s = np.asarray(slots_of(r), dtype=np.int64)
        wantO, wantL, tolO, tolL = L.attention(Q[r], values[np.maximum(s, 0)], s >= 0, scale)
        err = np.abs(O[r] - wantO)
        assert (err <= tolO).all(), f"row {r} of {len(s)}: O off {err.max():.3g}, {(err - tolO).max():.3g} over"
        if len(s[s >= 0]):
            err = np.abs(lse[r] - wantL)
            assert (err <= tolL).all(), f"row {r}: lse off {err.max():.3g}, allowed {tolL.min():.3g}"
        else:
            assert (lse[r] == -np.inf).all() and not O[r].any()


def _pages(lens, page, pages, seed):
    """A table with every row's pages in random order, and -1 beyond them."""
    rng = np.random.default_rng(seed)
    need = [-(-max(0, n) // page) for n in lens]
    order = rng.permutation(pages)
    assert sum(need) <= pages
    table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = order[at:at + k]
        at += k
    return table


def _decode_case(lens, nh, nope, pe, page, fmt, seed=0, scale=None, size=1.0):
    pages = sum(-(-max(0, n) // page) for n in lens) + 2
    cache, values = _pool(pages, page, nope, pe, fmt, seed)
    table = _pages(lens, page, pages, seed)
    q = _q(len(lens), nh, nope + pe, seed + 1, size)
    O, lse = ir.latent_attn_decode(q, cache, torch.from_numpy(table).cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda(), nope, pe, scale)
    assert O.shape == q.shape and O.dtype == torch.bfloat16 and lse.shape == q.shape[:2]
    t = np.arange(max(list(lens) + [0]))
    scale = (nope + pe) ** -0.5 if scale is None else scale
    _check(q, values, lambda r: table[r, t[:max(0, lens[r])] // page].astype(np.int64) * page
           + t[:max(0, lens[r])] % page, scale, O, lse)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("lens", [[1], [0], [2, 0, 1], [63], [64], [65], [127, 128, 129], [1000, 0, 0, 3, 257],
                                  [4097], [0, 0, 0], [5, 640, 64, 1, 320, 191]])
def test_decode_lengths(fmt, lens):
    _decode_case(lens, 64, 448, 64, 64, fmt, seed=sum(lens))


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("nh", [1, 2, 3, 15, 16, 17, 31, 33, 48, 63, 65, 80, 96, 127, 128])
def test_decode_heads(fmt, nh):
    _decode_case([130, 1, 700], nh, 448, 64, 64, fmt, seed=nh)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("nope,pe", [(480, 32), (96, 32), (64, 64), (48, 16), (16, 0), (16, 8), (512, 0), (112, 8),
                                     (256, 0), (272, 56), (368, 16), (16, 496)])
def test_decode_channel_splits(fmt, nope, pe):
    _decode_case([200, 77, 1], 20, nope, pe, 16, fmt, seed=nope)


@pytest.mark.parametrize("nope,pe", [(8, 0), (0, 8), (6, 2), (0, 64), (450, 62), (200, 56), (120, 0)])
def test_decode_channel_splits_of_bf16_rows(nope, pe):
    _decode_case([200, 77, 1], 20, nope, pe, 16, BF16, seed=nope)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("page", [1, 2, 7, 16, 48, 64, 100, 128, 1024])
def test_decode_page_sizes(fmt, page):
    _decode_case([300, 1, 129, 64], 16, 96, 32, page, fmt, seed=page)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_decode_one_long_row_and_a_batch_that_is_split(fmt):
    _decode_case([20011], 64, 448, 64, 64, fmt, seed=1)
    _decode_case([9000, 17, 4096, 0, 12345, 64, 1], 128, 448, 64, 16, fmt, seed=2)


def test_decode_many_short_rows():
    lens = [int(n) for n in np.random.default_rng(5).integers(0, 70, 1700)]
    _decode_case(lens, 5, 48, 16, 8, BF16, seed=3)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("nope,pe", [(48, 16), (128, 64), (320, 64), (448, 64)])
def test_decode_ragged_rows_of_every_block_count(fmt, nope, pe):
    """One to four blocks of 128 channels a tile: the ring's stages, and which
    warps fill them, fall differently on the tiles."""
    lens = [int(n) for n in np.random.default_rng(nope).integers(0, 400, 350)]
    _decode_case(lens, 9, nope, pe, 16, fmt, seed=nope)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("nh,nope,pe", [(128, 272, 16), (64, 448, 64), (40, 96, 32)])
def test_rows_between_empty_ones(fmt, nh, nope, pe):
    """A row without tokens has no tile, and so none of a tile's barriers: it must
    not touch what a slower warp still needs for the output of the row before."""
    for seed in range(6):
        rng = np.random.default_rng(seed)
        lens = [int(n) for n in rng.choice([0, 1, 1, 70, 200], 400, p=[0.5, 0.2, 0.2, 0.05, 0.05])]
        _decode_case(lens, nh, nope, pe, 8, fmt, seed=seed, size=0.2)


def test_groups_whose_scales_lie_far_apart():
    """Scales above 2^7 need two factors on the way to bf16; the queries are zero
    in the channels of large values, so that only the output shows them."""
    nope, pe, n, nh = 448, 64, 500, 20
    d, size = nope + pe, torch.ones(nope + pe)
    for group, e in enumerate([0, 20, 60, 100, -60, 8, 40]):
        size[64 * group:64 * group + 64] = 2.0 ** e
    x = (torch.randn(n, d, generator=torch.Generator().manual_seed(5)) * size).to(torch.bfloat16).cuda()
    cache = ir.kv_latent_empty(n, 1, nope, pe, E4M3)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    ir.kv_latent_write(cache, x, slots, nope, pe)
    values = f64(ir.kv_latent_read(cache, slots, nope, pe))
    assert (np.abs(values - f64(x)) <= np.abs(f64(x)) * 2.0 ** -4 + size.numpy() * 2.0 ** -8).all()
    q = _q(3, nh, d, 6) * (size <= 1.0).to(torch.bfloat16).cuda()
    O, lse = ir.latent_attn_sparse(q, cache, slots[None].repeat(3, 1).contiguous(), nope, pe, d ** -0.5)
    _check(q, values, lambda r: np.arange(n), d ** -0.5, O, lse)


@pytest.mark.parametrize("size,scale", [(1.0, 0.0), (30.0, None), (1.0, -0.3), (4.0, 2.0)])
def test_decode_scales_and_peaked_rows(size, scale):
    """Zero and negative scales, and scores large enough that the running
    maximum moves by far more than an exponential can hold."""
    _decode_case([900, 65, 3], 64, 448, 64, 64, BF16, seed=7, scale=scale, size=size)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_rising_scores_move_the_maximum_in_every_tile(fmt):
    nope, pe, n = 64, 64, 1500
    d = nope + pe
    x = torch.randn(n, d, generator=torch.Generator().manual_seed(0)) * 0.05
    x[:, 0] = torch.linspace(-3.0, 3.0, n)  # its product with q[0] = 64 rises from -192 to 192
    cache = ir.kv_latent_empty(n, 1, nope, pe, fmt)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    ir.kv_latent_write(cache, x.to(torch.bfloat16).cuda(), slots, nope, pe)
    values = f64(ir.kv_latent_read(cache, slots, nope, pe))
    q = _q(2, 3, d, 4)
    q[0, :, 0], q[1, :, 0] = 64.0, -64.0
    O, lse = ir.latent_attn_sparse(q, cache, slots[None].repeat(2, 1).contiguous(), nope, pe, 1.0)
    _check(q, values, lambda r: np.arange(n), 1.0, O, lse)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("rows,topk,nh", [(1, 1, 64), (3, 0, 8), (5, 2048, 64), (300, 130, 64), (40, 64, 128),
                                          (7, 65, 96), (2, 1000, 3), (200, 512, 16)])
def test_sparse(fmt, rows, topk, nh):
    nope, pe, page = 448, 64, 64
    cache, values = _pool(40, page, nope, pe, fmt, rows + topk)
    rng = np.random.default_rng(topk)
    idx = rng.integers(0, 40 * page, (rows, topk)).astype(np.int32)  # repeats are counted each time
    idx[rng.random((rows, topk)) < 0.05] = -1
    if rows > 2 and topk:
        idx[1] = -1                      # a row with nothing
        idx[2, : topk // 2] = -5         # a long left-out head
        idx[0, topk // 2:] = 2**31 - 1   # and tail
    q = _q(rows, nh, 512, rows)
    O, lse = ir.latent_attn_sparse(q, cache, torch.from_numpy(idx).cuda(), nope, pe)
    ok = (idx >= 0) & (idx < 40 * page)
    _check(q, values, lambda r: np.where(ok[r], idx[r], -1), 512 ** -0.5, O, lse)


def test_sparse_over_the_remapped_table():
    """Batch-local indices, made flat-global by the remap, select the rows."""
    nope, pe, b, sq, skv, topk = 96, 32, 3, 4, 160, 50
    cache, values = _pool(b * skv // 16, 16, nope, pe, E4M3, 8)
    rng = np.random.default_rng(8)
    local = rng.integers(-1, skv, (b * sq, topk)).astype(np.int32)
    idx = ir.kv_idx_local_to_global(torch.from_numpy(local).cuda(), sq, skv)
    q = _q(b * sq, 10, 128, 9)
    O, lse = ir.latent_attn_sparse(q, cache, idx, nope, pe)
    _check(q, values, lambda r: np.where(local[r] >= 0, local[r] + (r // sq) * skv, -1), 128 ** -0.5, O, lse)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_bad_pages_and_lengths_are_left_out(fmt):
    nope, pe, page, pages = 448, 64, 16, 20
    cache, values = _pool(pages, page, nope, pe, fmt, 11)
    table = np.array([[3, -1, 5, 20, 7], [2**31 - 1, -2**31, 1, 2, 19], [0, 1, 2, 3, 4], [4, 3, 2, 1, 0],
                      [-1, -1, -1, -1, -1]], np.int32)
    lens = np.array([75, 80, -5, 2**31 - 1, 80], np.int32)
    q = _q(5, 64, 512, 12)
    O, lse = ir.latent_attn_decode(q, cache, torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(), nope, pe)

    def slots(r):
        t = np.arange(min(max(0, int(lens[r])), 80))
        pg = table[r, t // page].astype(np.int64)
        return np.where((pg >= 0) & (pg < pages), pg * page + t % page, -1)
    _check(q, values, slots, 512 ** -0.5, O, lse)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_rows_that_are_not_attended_to_may_hold_anything(fmt):
    """NaN and infinities in the rest of the last page, in other pages, beyond
    the table and in another row's tokens."""
    nope, pe, page = 448, 64, 32
    cache, values = _pool(30, page, nope, pe, fmt, 13)
    lens = [33, 1, 100]
    table = _pages(lens, page, 30, 13)
    used = np.zeros(30 * page, bool)
    for r, n in enumerate(lens):
        t = np.arange(n)
        used[table[r, t // page] * page + t % page] = True
    flat = cache.view(30 * page, -1)
    junk = torch.from_numpy(~used).cuda()
    flat.view(torch.uint8)[junk] = 0xFF  # bf16 NaN; scale byte 255
    q = _q(3, 64, 512, 14)
    args = (torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), nope, pe)
    O, lse = ir.latent_attn_decode(q, cache, *args)
    t = np.arange(100)
    _check(q, values, lambda r: table[r, t[:lens[r]] // page] * page + t[:lens[r]] % page, 512 ** -0.5, O, lse)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_nan_and_infinity_show_where_they_reach(fmt):
    nope, pe, page, nh = 448, 64, 16, 64
    cache, values = _pool(30, page, nope, pe, fmt, 15)
    table = torch.arange(30, dtype=torch.int32, device="cuda").view(3, 10).contiguous()
    lens = torch.tensor([150, 150, 150], dtype=torch.int32, device="cuda")
    q = _q(3, nh, 512, 16)
    O0, lse0 = ir.latent_attn_decode(q, cache, table, lens, nope, pe)
    q2 = q.clone()
    q2[0, 5, 100] = float("nan")
    x = torch.full((1, 512), 1.0, dtype=torch.bfloat16, device="cuda")
    x[0, 3] = float("nan")
    ir.kv_latent_write(cache, x, torch.tensor([10 * page + 7], dtype=torch.int32, device="cuda"), nope, pe)
    O, lse = ir.latent_attn_decode(q2, cache, table, lens, nope, pe)
    assert torch.isnan(O[0, 5]).all() and torch.isnan(lse[0, 5])
    keep = [h for h in range(nh) if h != 5]
    assert torch.equal(O[0, keep], O0[0, keep]) and torch.equal(lse[0, keep], lse0[0, keep])
    assert torch.isnan(lse[1]).all() and torch.isnan(O[1]).all()
    assert torch.equal(O[2], O0[2])


def test_cache_beyond_four_gigabytes():
    nope, pe, page = 448, 64, 64
    pages = 5 * 2**20 // page
    cache = ir.kv_latent_empty(pages, page, nope, pe, BF16)
    assert cache.numel() * 2 > 2**32
    x = torch.randn(256, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    at = torch.arange((pages - 4) * page, pages * page, dtype=torch.int32, device="cuda")
    ir.kv_latent_write(cache, x.cuda(), at, nope, pe)
    q = _q(1, 64, 512, 2)
    table = torch.tensor([[pages - 1, pages - 4, pages - 2]], dtype=torch.int32, device="cuda")
    O, lse = ir.latent_attn_decode(q, cache, table, torch.tensor([150], dtype=torch.int32, device="cuda"), nope, pe)
    order = np.concatenate([np.arange(192, 256), np.arange(0, 64), np.arange(128, 150)])
    _check(q, f64(x), lambda r: order, 512 ** -0.5, O, lse)


def test_same_bits_every_time_and_a_dirty_workspace():
    nope, pe, rows, nh = 448, 64, 5, 128
    cache, _ = _pool(200, 64, nope, pe, E4M3, 17)
    table = torch.arange(200, dtype=torch.int32, device="cuda").view(5, 40).contiguous()
    lens = torch.tensor([2500, 1, 0, 777, 2000], dtype=torch.int32, device="cuda")
    q = _q(rows, nh, 512, 18)
    nbytes = ir.latent_attn_workspace_bytes(rows, nh, 40 * 64, nope, pe)
    ws = torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")
    ref = None
    for fill in (0, 0xFF, 0x7F, 3):
        ws.fill_(fill)
        O, lse = ir.latent_attn_decode(q, cache, table, lens, nope, pe, workspace=ws)
        if ref is None:
            ref = O, lse
        assert torch.equal(O, ref[0]) and torch.equal(lse, ref[1])
    O, lse = ir.latent_attn_decode(q, cache, table, lens, nope, pe)
    assert torch.equal(O, ref[0]) and torch.equal(lse, ref[1])
    if nbytes:
        with pytest.raises(ir.InvropeError, match="WORKSPACE"):
            ir.latent_attn_decode(q, cache, table, lens, nope, pe, workspace=ws[:nbytes - 16])


def test_streams_and_graph():
    """Calls on two streams at once, and a captured call whose lengths, pages
    and queries change between replays."""
    nope, pe, nh = 448, 64, 64
    cache, values = _pool(120, 64, nope, pe, BF16, 19)
    table = torch.arange(120, dtype=torch.int32, device="cuda").view(3, 40).contiguous()
    cases = [(_q(3, nh, 512, 20 + k), torch.tensor(n, dtype=torch.int32, device="cuda"))
             for k, n in enumerate([[2000, 5, 700], [1, 2560, 64], [0, 0, 9]])]
    ref = [ir.latent_attn_decode(q, cache, table, n, nope, pe) for q, n in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[ir.latent_attn_decode(q, cache, table, n, nope, pe, stream=s) for (q, n), s in zip(cases, streams)]
           for _ in range(4)]
    torch.cuda.synchronize()
    for step in got:
        for (O, lse), (O0, lse0) in zip(step, ref):
            assert torch.equal(O, O0) and torch.equal(lse, lse0)
    q, n = cases[0][0].clone(), cases[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, lse = ir.latent_attn_decode(q, cache, table, n, nope, pe)
    for (q1, n1), (O0, lse0) in zip(cases, ref):
        q.copy_(q1)
        n.copy_(n1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, O0) and torch.equal(lse, lse0)


def test_outputs_given_and_no_rows():
    nope, pe = 96, 32
    cache, values = _pool(10, 16, nope, pe, BF16, 21)
    q = _q(2, 6, 128, 22)
    idx = torch.arange(160, dtype=torch.int32, device="cuda").view(2, 80).contiguous()
    O, lse = torch.empty_like(q), torch.empty(2, 6, device="cuda")
    a, b = ir.latent_attn_sparse(q, cache, idx, nope, pe, O=O, lse=lse)
    assert a is O and b is lse
    _check(q, values, lambda r: np.arange(80) + 80 * r, 128 ** -0.5, O, lse)
    O, lse = ir.latent_attn_sparse(q[:0], cache, idx[:0], nope, pe)
    assert O.shape == (0, 6, 128) and lse.shape == (0, 6)
    with pytest.raises(ir.InvropeError, match="INVALID"):
        ir.latent_attn_sparse(q, cache, idx, nope, pe, O=q)


def test_output_goes_into_the_postmix():
    """The step after: inverse rotation of the pe channels and the head mix."""
    nope, pe, nh, rows = 448, 64, 64, 4
    cache, values = _pool(20, 64, nope, pe, E4M3, 23)
    q = _q(rows, nh, 512, 24)
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(4, 5).contiguous()
    lens = torch.tensor([320, 100, 1, 64], dtype=torch.int32, device="cuda")
    O, _ = ir.latent_attn_decode(q, cache, table, lens, nope, pe)
    M = torch.eye(nh, device="cuda")
    Y = ir.invrope_postmix_fwd_ex(O, M, nope, pe, positions=lens - 1)
    torch.cuda.synchronize()
    import oracle
    want = oracle.postmix_fwd(f64(O), f64(M), (lens - 1).cpu().numpy().astype(np.int64), nope, pe, 10000.0)
    assert np.abs(f64(Y) - want).max() <= 8e-3 * np.abs(want).max()
