"""Token numbers to slots where a sequence's page table goes through shared memory: tables
of many rows a sequence, every entry against plain indexing. Needs a GB300."""

import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _rows(topk):
    """The fewest rows of a sequence for which its table is staged: 16 chunks of 2048 vectors
    (four entries, or one where rows are no vectors) for each multiprocessor."""
    vectors = 16 * 1024 * torch.cuda.get_device_properties(0).multi_processor_count
    return -(-vectors // (topk // 4 if topk % 4 == 0 else topk))


def _want(idx, table, lens, page, pages, seq):
    seqs, width = table.shape
    known = (seq >= 0) & (seq < seqs)
    s = torch.where(known, seq, 0)
    end = torch.where(known, lens.long().clamp(max=width * page)[s], 0)
    token = idx.long()
    ok = (token >= 0) & (token < end[:, None])
    token = torch.where(ok, token, 0)
    held = table.long()[s[:, None], token // page]
    return torch.where(ok & (held >= 0) & (held < pages), held * page + token % page, -1).int()


def _inputs(rows, topk, seqs, width, page, seed, lens=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ints = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)  # noqa: E731
    pages = seqs * width
    table = ints(-2, pages + 2, seqs, width)
    lens = ints(width * page // 2, width * page + 20, seqs) if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    idx = ints(-5, width * page + 30, rows, topk)
    idx[0, 0], idx[-1, -1] = 2**31 - 1, -2**31
    return idx, table, lens, pages


def _staged(call):
    """Whether `call` launched the staged kernel (None where the profiler says nothing: a
    process's first profile may be empty)."""
    from torch.profiler import ProfilerActivity, profile
    for _ in range(3):
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            call()
            torch.cuda.synchronize()
        names = " ".join(e.key for e in prof.key_averages())
        if "slots_" in names:
            return "slots_staged_kernel" in names
    return None


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("topk,more,seqs,gone,width,page", [
    (2048, 0, 2, 0, 300, 64),    # exactly as many vectors as it takes; chunks of whole rows
    (2052, 1, 3, 0, 100, 48),    # chunks over two sequences' rows
    (2052, 5, 3, 1, 8192, 1),    # the longest table, and rows behind the last sequence
    (641, 0, 2, 0, 256, 64),     # rows that are no vectors
    (641, 3, 3, 1, 8192, 3),
    (65537, 0, 2, 0, 100, 16),   # rows of more than a chunk
    (3, 1, 2, 0, 7, 5),          # chunks of many rows
])
def test_every_entry(topk, more, seqs, gone, width, page, in_place):
    sq = _rows(topk) + more
    rows = seqs * sq - sq // 3
    idx, table, lens, pages = _inputs(rows, topk, seqs - gone, width, page, topk + width)
    want = _want(idx, table, lens, page, pages, torch.arange(rows, device="cuda") // sq)
    got = ir.kv_idx_local_to_slots(idx, table, lens, page, pages, sq, out=idx if in_place else None)
    assert torch.equal(got, want)


@pytest.mark.parametrize("topk", [2048, 641])
def test_lengths_without_a_token_and_beyond_the_table(topk):
    sq, width, page = _rows(topk), 50, 64
    lens = [0, 2**31 - 1, -2**31, 1, 3200]
    idx, table, lens, pages = _inputs(5 * sq, topk, 5, width, page, topk, lens)
    got = ir.kv_idx_local_to_slots(idx, table, lens, page, pages, sq)
    assert torch.equal(got, _want(idx, table, lens, page, pages, torch.arange(5 * sq, device="cuda") // sq))


@pytest.mark.parametrize("topk,more,width,staged", [(2048, 0, 8192, True), (2048, -1, 8192, False), (2048, 0, 8193, False),
                                                    (641, 0, 8192, True), (641, -1, 8192, False), (641, 0, 8193, False)])
def test_where_the_table_is_staged(topk, more, width, staged):
    """Both sides of each limit give the plain result, and the cases above run what they are for."""
    sq = _rows(topk) + more
    idx, table, lens, pages = _inputs(2 * sq, topk, 2, width, 2, width)
    got = []
    ran = _staged(lambda: got.append(ir.kv_idx_local_to_slots(idx, table, lens, 2, pages, sq)))
    assert torch.equal(got[-1], _want(idx, table, lens, 2, pages, torch.arange(2 * sq, device="cuda") // sq))
    assert ran in (staged, None)


@pytest.mark.parametrize("sq", [2**31 - 1, 2**31, 2**40, 2**60, 2**61, 2**62, 2**63 - 1])
@pytest.mark.parametrize("topk", [16, 641])
def test_more_rows_a_sequence_than_there_are(topk, sq):
    """All rows are of the first sequence. A product of sq with a row's four vectors would not
    fit 64 bits."""
    rows = 2 * _rows(topk)
    idx, table, lens, pages = _inputs(rows, topk, 2, 40, 64, 9)
    got = []
    ran = _staged(lambda: got.append(ir.kv_idx_local_to_slots(idx, table, lens, 64, pages, sq)))
    assert torch.equal(got[-1], _want(idx, table, lens, 64, pages, torch.zeros(rows, dtype=torch.long, device="cuda")))
    assert ran is not False


def test_replayed_and_on_another_stream():
    topk, width, page = 2052, 100, 48
    sq = _rows(topk)
    idx, table, lens, pages = _inputs(2 * sq, topk, 2, width, page, 4)
    seq, out = torch.arange(2 * sq, device="cuda") // sq, torch.empty_like(idx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ir.kv_idx_local_to_slots(idx, table, lens, page, pages, sq, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = ir.kv_idx_local_to_slots(idx, table, lens, page, pages, sq, stream=side)
    side.synchronize()
    assert torch.equal(there, _want(idx, table, lens, page, pages, seq))
    lens.fill_(777)
    table.copy_(table.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _want(idx, table, lens, page, pages, seq))
