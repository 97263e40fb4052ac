"""Serve synthetic sequences from a latent cache: the library's operators in the
order in which a decoder layer calls them.

    python -m partial_inverse_rope_gb300.run_decode --rows 8 --prompt 4096 --steps 16 --fmt e4m3
    python -m partial_inverse_rope_gb300.run_decode --rows 32 --prompt 16384 --steps 64 --graph
    python -m partial_inverse_rope_gb300.run_decode --rows 32 --prompt 16384 --fmt e2m1 --pool --graph

Prompt: the tokens' latent vectors go into the cache (``kv_latent_write``). The
last ``--chunk`` tokens of each sequence attend to ``--topk`` selected ones
each: the batch-local table becomes flat-global (``kv_idx_local_to_global``),
and ``latent_attn_sparse`` reads the rows that it names.

Step: one new vector a sequence is appended, ``latent_attn_decode`` attends to
all of its tokens through the page table, and the attention's output, whose pe
channels are still rotated by the position, goes through the inverse rotation
and the head mix (``invrope_postmix_fwd_ex`` at each row's own position). Page
table, lengths, slots and positions stay on the device; with --graph a step is
captured once and replayed.

With --pool the sequences share a pool of pages, three quarters of what they could
fill, or what their prompts need where that is more: ``kv_pages_advance`` hands out
pages, slots and positions and takes pages back when a sequence ends, and ``rope_apply``
turns queries and vectors by their positions, in front of what the postmix turns back.
Halfway through, and at the end, every fourth sequence ends and begins again with a
prompt. The last line says how many prompts and how many of the steps' tokens found no page.

The process exits non-zero if a kernel's watchdog fired, an output is not finite, or a
prompt was refused.
"""

from __future__ import annotations

import argparse
import sys

import torch

from . import binding as ir
from . import inputs as W


class Server:
    """A batch of sequences over one layer's cache. Sequence r owns the pages
    [r * pages, (r + 1) * pages), so its token t has slot r * capacity + t. It holds
    ``capacity`` tokens: a longer prompt is refused, and in a full sequence the
    newest token takes the last one's place, at its own position. ``lens`` counts
    all tokens, on the device, where a replayed graph reads it."""

    def __init__(self, rows, capacity, nh, nope, pe, page, fmt, seed=0, device="cuda"):
        pages = -(-capacity // page)
        self.rows, self.nh, self.nope, self.pe, self.d = rows, nh, nope, pe, nope + pe
        self.capacity = pages * page
        self.cache = ir.kv_latent_empty(rows * pages, page, nope, pe, fmt, device=device)
        self.table = torch.arange(rows * pages, dtype=torch.int32, device=device).view(rows, pages)
        self.first = torch.arange(rows, dtype=torch.int32, device=device) * self.capacity
        # lengths and the next tokens' slots, with what they stay below, and a copy for a step
        self.state = torch.stack([torch.zeros_like(self.first), self.first])
        self.most = torch.stack([torch.full_like(self.first, 2**31 - 2), self.first + (self.capacity - 1)])
        self.now = self.state.clone()
        self.lens, self.positions, self.slots = self.state[0], self.now[0], self.now[1]
        self.M = W.postmix_M(nh, seed, device=device)

    def prompt(self, x, lens):
        """Vectors ``x`` [sum(lens), d], sequence after sequence."""
        if int(lens.max()) > self.capacity:
            raise ValueError(f"a prompt has {int(lens.max())} tokens, a sequence holds {self.capacity}")
        torch.minimum(torch.stack([lens.int(), self.first + lens.int()]), self.most, out=self.state)
        which = torch.repeat_interleave(torch.arange(self.rows, device=x.device), lens.long())
        begin = torch.cumsum(lens.long(), 0) - lens
        slots = which * self.capacity + torch.arange(len(x), device=x.device) - begin[which]
        ir.kv_latent_write(self.cache, x, slots.int(), self.nope, self.pe)

    def selected(self, q, idx, positions):
        """Queries [rows * chunk, nh, d] over batch-local ``idx`` [rows * chunk,
        topk] (-1: none); returns the mixed output."""
        table = ir.kv_idx_local_to_global(idx, len(idx) // self.rows, self.capacity)
        O, _ = ir.latent_attn_sparse(q, self.cache, table, self.nope, self.pe)
        return ir.invrope_postmix_fwd_ex(O, self.M, self.nope, self.pe, positions=positions)

    def step(self, x, q):
        """One token a sequence: its vector ``x`` [rows, d] and queries ``q``
        [rows, nh, d]; returns the mixed output [rows, nh, d]."""
        self.now.copy_(self.state)
        self.state += 1
        torch.minimum(self.state, self.most, out=self.state)
        ir.kv_latent_write(self.cache, x, self.slots, self.nope, self.pe)
        O, _ = ir.latent_attn_decode(q, self.cache, self.table, self.lens, self.nope, self.pe)
        return ir.invrope_postmix_fwd_ex(O, self.M, self.nope, self.pe, positions=self.positions)


class PooledServer:
    """A batch of sequences over one layer's cache whose pages are of one pool. A
    sequence that gets no page keeps its tokens and has not taken the step: ``granted``
    int32 [rows] says after each step who has (1) and who has not (0). All state is on the
    device, where a replayed graph advances it, ``granted`` too."""

    def __init__(self, rows, capacity, pages, nh, nope, pe, page, fmt, seed=0, device="cuda"):
        self.rows, self.nh, self.nope, self.pe, self.page, self.d = rows, nh, nope, pe, page, nope + pe
        self.cache = ir.kv_latent_empty(pages, page, nope, pe, fmt, device=device)
        self.state, self.table, self.queue = ir.kv_pages_empty(rows, -(-capacity // page), pages, device=device)
        self.lens = self.state[:rows]
        self.freqs, _ = ir.rope_freqs(pe)
        self.one = torch.ones(rows, dtype=torch.int32, device=device)
        # what a step's call gives: one place for all steps, so that a replayed one's is known
        self.out = tuple(torch.zeros(n, dtype=torch.int32, device=device) for n in (rows, rows, rows, rows + 1, rows))
        self.slots, self.positions, _, _, self.granted = self.out
        self.M = W.postmix_M(nh, seed, device=device)

    def prompt(self, x, new):
        """Vectors ``x`` [tokens, d] for the sequences that ``new`` int32 [rows] has tokens of,
        one after the other; a negative number ends a sequence. Returns how many each got."""
        slots, positions, _, _, granted = ir.kv_pages_advance(self.state, self.table, self.queue, new, self.page, len(x))
        ir.kv_latent_write(self.cache, ir.rope_apply(x, self.freqs, positions), slots, self.nope, self.pe)
        return granted

    def step(self, x, q):
        """One token a sequence: its vector ``x`` [rows, d] and queries ``q`` [rows, nh, d];
        returns the mixed output [rows, nh, d]. Where ``granted`` is 0 afterwards the vector is
        not in the cache and the row of the output answers no query (its place in the sequence
        is not known to the call, which works at position 0 there): the sequence's step is to be
        asked for again when others have given pages back."""
        ir.kv_pages_advance(self.state, self.table, self.queue, self.one, self.page, self.rows, out=self.out)
        q, x = ir.rope_apply([q, x], self.freqs, self.positions)
        ir.kv_latent_write(self.cache, x, self.slots, self.nope, self.pe)
        O, _ = ir.latent_attn_decode(q, self.cache, self.table, self.lens, self.nope, self.pe)
        return ir.invrope_postmix_fwd_ex(O, self.M, self.nope, self.pe, positions=self.positions)

    def selected(self, q, idx, positions):
        """Queries [rows * chunk, nh, d] over token numbers ``idx`` [rows * chunk, topk] of their
        own sequence (-1: none); returns the mixed output."""
        slots = ir.kv_idx_local_to_slots(idx, self.table, self.lens, self.page, len(self.queue), len(idx) // self.rows)
        O, _ = ir.latent_attn_sparse(ir.rope_apply(q, self.freqs, positions), self.cache, slots, self.nope, self.pe)
        return ir.invrope_postmix_fwd_ex(O, self.M, self.nope, self.pe, positions=positions)


def pool_pages(lens, most, page):
    """Pages of a pool for sequences with prompts of these lengths and up to ``most`` tokens:
    three quarters of what they could fill, and no fewer than the prompts and a first new
    page of each take."""
    return max(-(-3 * len(lens) * -(-most // page) // 4), sum(-(-n // page) + 1 for n in lens))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=8, help="sequences")
    ap.add_argument("--prompt", type=int, default=4096, help="longest prompt; lengths are spread down to half of it")
    ap.add_argument("--chunk", type=int, default=16, help="prompt tokens a sequence that attend to selected ones")
    ap.add_argument("--topk", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--nh", type=int, default=64)
    ap.add_argument("--nope", type=int, default=448)
    ap.add_argument("--pe", type=int, default=64)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--fmt", choices=["bf16", "e4m3", "e2m1"], default="e4m3")
    ap.add_argument("--pool", action="store_true", help="pages of one pool, rotary positions")
    ap.add_argument("--graph", action="store_true", help="capture one step and replay it")
    args = ap.parse_args(argv)
    if args.prompt < 1:
        ap.error("--prompt must be at least 1: a selected token has to have been written")

    dev, d = torch.device("cuda", 0), args.nope + args.pe
    fmt = {"bf16": ir.KV_LATENT_BF16, "e4m3": ir.KV_LATENT_E4M3, "e2m1": ir.KV_LATENT_E2M1}[args.fmt]
    most = args.prompt + args.steps + 4
    lens = torch.linspace(max(1, args.prompt // 2), args.prompt, args.rows, device=dev).int()
    if args.pool:
        server = PooledServer(args.rows, most, pool_pages(lens.tolist(), most, args.page), args.nh, args.nope, args.pe,
                              args.page, fmt, device=dev)
    else:
        server = Server(args.rows, most, args.nh, args.nope, args.pe, args.page, fmt, device=dev)

    refused = dropped = 0  # prompts and tokens of steps that found no page
    taken = server.prompt(W.normal_bf16((int(lens.sum()), d), 1, device=dev), lens)
    if args.pool:
        refused += int((taken != lens).sum())
    rows = args.rows * args.chunk
    idx = (torch.rand(rows, args.topk, device=dev) * lens.repeat_interleave(args.chunk)[:, None]).int()
    at = (lens[:, None] - args.chunk + torch.arange(args.chunk, device=dev)).clamp_min(0).int().flatten()
    idx = torch.where(idx <= at[:, None], idx, -1)  # causal
    Y = server.selected(W.normal_bf16((rows, args.nh, d), 2, device=dev), idx.contiguous(), at)
    finite = bool(torch.isfinite(Y).all())

    x, q = W.normal_bf16((args.rows, d), 3, device=dev), W.normal_bf16((args.rows, args.nh, d), 4, device=dev)
    step = lambda: server.step(x, q)
    for _ in range(3):
        Y = step()
    if args.graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Y = step()
        step = graph.replay
    us = 0.0
    for part in ((args.steps // 2, args.steps - args.steps // 2) if args.pool else (args.steps,)):
        before = int(server.lens.sum())
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        e0.record()
        for _ in range(part):
            out = step()  # (a replay returns nothing and leaves its output in Y)
            Y = Y if args.graph else out
        e1.record()
        torch.cuda.synchronize()
        us += e0.elapsed_time(e1) * 1e3
        if args.pool:
            dropped += part * args.rows - (int(server.lens.sum()) - before)
            gone = torch.arange(args.rows, device=dev) % 4 == 0
            server.prompt(x[:0], torch.where(gone, -1, 0).int())
            again = torch.where(gone, lens, 0).int()
            refused += int((server.prompt(W.normal_bf16((int(lens[gone].sum()), d), 5, device=dev), again) != again).sum())
    finite = finite and bool(torch.isfinite(Y).all())
    us /= max(1, args.steps)
    fault = ir.invrope_take_device_fault()
    print(f"{args.rows} sequences of {int(server.lens.min())} to {int(server.lens.max())} tokens, {args.fmt} cache: "
          f"{us:.1f} us a step{' (graph)' if args.graph else ''}; outputs finite: {finite}; "
          f"watchdog fault code {fault}"
          + (f"; no page for {refused} prompts and {dropped} of {args.steps * args.rows} tokens" if args.pool else ""))
    return 1 if fault or not finite or refused else 0


if __name__ == "__main__":
    sys.exit(main())
