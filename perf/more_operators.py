"""Measured cases of what stands around the latent cache in a serving or training
step: positions, pages, and a cache held in 4 bits.

* ``rope``: rotary positions on all or the last channels of each head, in the half
  or the interleaved layout, forward or as its gradient.
* ``pages``: one step of a batch of sequences over a paged cache: pages are handed
  out and taken back, and every new token gets its slot and its position.
* ``slots``: token numbers within a sequence become cache slots, through its pages.
* ``cache``: vectors are written into a cache of 4-bit rows and read back, or rows
  are read.
* ``attend``: attention over such a cache, a sequence's pages or selected rows.

``own`` chooses between elementary torch operations and the package's kernels.

A 4-bit row is ``nope / 2`` bytes of e2m1 codes, ``pe`` bf16 values, one power-of-two
scale byte (biased by 127) for each 32 codes, and padding to 16 bytes. Four bytes
hold 8 channels: channel 2p + h has the bits 16h + 4p and on.
"""

import math

import torch

own = False

GROUP = 32          # channels that share a scale
E_MIN, E_MAX = -126, 125


def listed():
    base = {"nope": 448, "pe": 64}
    return [
        # one decoding step of 64 sequences: their queries and their new latent vectors
        {"name": "rope_64_decode", "op": "rope", "n": 64, "nh": 64, "d": 512, "pe": 64, "type": "bf16", "inter": False,
         "back": False, "latent": True, "factor": 1.0},
        # the queries of a prompt shard of 16384 tokens, far into the context
        {"name": "rope_16384_prompt", "op": "rope", "n": 16384, "nh": 64, "d": 512, "pe": 64, "type": "bf16", "inter": False,
         "back": False, "latent": False, "factor": 1.0},
        # the gradient of whole heads in fp32, interleaved, in a context extended four times
        {"name": "rope_10007_grad_fp32", "op": "rope", "n": 10007, "nh": 48, "d": 128, "pe": 128, "type": "fp32", "inter": True,
         "back": True, "latent": False, "factor": 4.0},
        # one decoding step of 64 sequences: one token each
        {"name": "pages_64_decode", "op": "pages", "rows": 64, "prompts": 0, "chunk": 1, "gone": 0, "page": 64,
         "max_pages": 256, "free": 64},
        # a large batch: decoding rows, prompt chunks and sequences that ended
        {"name": "pages_1000_mixed", "op": "pages", "rows": 1000, "prompts": 40, "chunk": 4096, "gone": 31, "page": 64,
         "max_pages": 1024, "free": 1700},
        # selected tokens of 64 decoding rows
        {"name": "slots_64x2048", "op": "slots", "rows": 64, "sq": 1, "topk": 2048, "len": 65536, "page": 64},
        # the table of a prompt shard: 4 sequences of 16384 rows
        {"name": "slots_65536x2048", "op": "slots", "rows": 65536, "sq": 16384, "topk": 2048, "len": 16384, "page": 64},
        # one decoding step of 64 sequences puts one token each into the cache
        {"name": "append_64", "op": "cache", "write": True, "n": 64, "pages": 2048, "page": 64, **base},
        # the whole of a 64K context, for a prompt that continues it
        {"name": "read_65536", "op": "cache", "write": False, "n": 65536, "pages": 2048, "page": 64, **base},
        # an ordinary serving batch, ragged
        {"name": "decode_32_ragged", "op": "attend", "picked": False, "rows": 32, "nh": 64, "lo": 1, "hi": 16384, "page": 64, **base},
        # a large batch
        {"name": "decode_96_ragged", "op": "attend", "picked": False, "rows": 96, "nh": 64, "lo": 4000, "hi": 20000, "page": 64, **base},
        # a prompt chunk, every row with its own selection
        {"name": "sparse_2048x2048", "op": "attend", "picked": True, "rows": 2048, "nh": 64, "topk": 2048, "slots": 65536, "page": 64, **base},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "pages", "slots", "cache", "attend", "attend"])
    page = rng.choice([1, 16, 48, 64, 64, 128])
    if op == "rope":
        d, pe = rng.choice([(512, 64), (512, 64), (128, 128), (192, 64), (128, 32), (64, 64), (96, 10), (256, 128)])
        nh = rng.choice([1, 3, 8, 48, 64, 128])
        return {"op": op, "n": _spread(rng, 1, max(2, min(131072, (1 << 28) // (nh * d)))), "nh": nh, "d": d, "pe": pe,
                "type": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "inter": rng.random() < 0.4,
                "back": rng.random() < 0.4, "latent": rng.random() < 0.3, "factor": rng.choice([1.0, 1.0, 4.0, 40.0])}
    if op == "pages":
        rows, page = _spread(rng, 1, 4096), rng.choice([16, 48, 64, 128])
        prompts = rng.randint(0, min(rows, 64))
        chunk = _spread(rng, 1, 2048)
        most = prompts * (chunk // page + 2) + rows // page + 8
        return {"op": op, "rows": rows, "prompts": prompts, "chunk": chunk, "gone": rng.randint(0, (rows - prompts) // 2),
                "page": page, "max_pages": rng.choice([64, 256, 1024]), "free": rng.randint(1, 2 * most)}
    if op == "slots":
        rows, sq = _spread(rng, 1, 16384), _spread(rng, 1, 4096)
        return {"op": op, "rows": rows, "sq": sq, "topk": _spread(rng, 1, 4096), "len": _spread(rng, 1, 65536), "page": page}
    nope, pe = rng.choice([(448, 64), (448, 64), (96, 32), (64, 64), (480, 32), (32, 16), (512, 0)])
    if op == "cache":
        write = rng.random() < 0.5
        n = _spread(rng, 1, 16384 if write else 65536)
        return {"op": op, "write": write, "n": n, "pages": -(-max(4 * n, 4096) // page), "page": page, "nope": nope, "pe": pe}
    case = {"op": op, "nh": rng.choice([1, 3, 16, 48, 64, 64, 96, 128]), "page": page, "nope": nope, "pe": pe}
    if rng.random() < 0.6:
        rows = _spread(rng, 1, 128)
        hi = _spread(rng, 1, min(65536, 1 << 20) // max(1, rows // 16))
        return {**case, "picked": False, "rows": rows, "lo": rng.randint(0, hi), "hi": hi}
    return {**case, "picked": True, "rows": _spread(rng, 1, 1024), "topk": _spread(rng, 1, 2048), "slots": _spread(rng, 2048, 65536)}


def _row_bytes(nope, pe):
    return -(-(nope // 2 + 2 * pe + nope // GROUP) // 16) * 16


def _lens(case):
    """Lengths from lo to hi in even steps: the same total whatever the seed."""
    r = case["rows"]
    return [case["hi"] if r == 1 else case["lo"] + (case["hi"] - case["lo"]) * i // (r - 1) for i in range(r)]


def _asked(case):
    """Tokens that the sequences of a step ask for, in any order: chunks of prompts, -1 for
    those that ended, and one token for each of the others."""
    p, gone = case["prompts"], case["gone"]
    return [max(1, case["chunk"] * (i + 1) // p) for i in range(p)] + [-1] * gone + [1] * (case["rows"] - p - gone)


def _room(case):
    """Tokens that the step's arrays hold: a little more than are asked for."""
    return -(-sum(max(0, n) for n in _asked(case)) // 64) * 64 or 64


_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    if case["op"] == "rope":
        vectors = case["n"] * (case["nh"] + (1 if case["latent"] else 0))
        return {"bytes": 2 * vectors * case["d"] * _BYTES[case["type"]] + 4 * case["n"], "flops": 3 * vectors * case["pe"]}
    if case["op"] == "pages":
        # a sequence: tokens asked for, length in and out, granted, start; a token: slot, position, row; a page
        # that is handed out: from the queue into the table
        pages = sum(-(-n // case["page"]) for n in _asked(case) if n > 1)
        return {"bytes": 20 * case["rows"] + 12 * _room(case) + 8 * min(pages, case["free"]), "flops": 0}
    if case["op"] == "slots":
        seqs = -(-case["rows"] // case["sq"])
        return {"bytes": 8 * case["rows"] * case["topk"] + 4 * seqs * (-(-case["len"] // case["page"]) + 1), "flops": 0}
    nope, pe = case["nope"], case["pe"]
    d, rb = nope + pe, _row_bytes(nope, pe)
    if case["op"] == "cache":
        # rows in, vectors out, slots; a write before it: vectors in, rows out, slots
        return {"bytes": case["n"] * (rb + 2 * d + 4) * (2 if case["write"] else 1), "flops": 0}
    rows, nh = case["rows"], case["nh"]
    io = rows * nh * (4 * d + 4)  # queries in, outputs and log-sum-exp out
    if not case["picked"]:
        tokens = sum(_lens(case))
        table = 4 * sum(-(-n // case["page"]) for n in _lens(case))
        return {"bytes": tokens * rb + io + table + 4 * rows, "flops": 4 * tokens * nh * d}
    picked = rows * case["topk"]
    return {"bytes": min(picked, case["slots"]) * rb + io + 4 * picked, "flops": 4 * picked * nh * d}


# ---------------------------------------------------------------- the cache's rows

def _pow2(e):
    """2^e for whole e from -126 to 127, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x, nope, pe):
    """bf16 vectors [n, d] -> cache rows uint8 [n, row bytes]."""
    n = x.shape[0]
    v = x[:, :nope].float().view(n, nope // GROUP, GROUP)
    mant, exp = torch.frexp(v.abs().amax(-1))
    e = torch.where(mant <= 0.75, exp - 3, exp - 2).clamp(E_MIN, E_MAX)  # the least e with amax <= 6 * 2^e
    bad = ~torch.isfinite(v).all(-1)
    e = torch.where(bad, torch.zeros_like(e), e)
    v = torch.where(bad[..., None], torch.zeros_like(v), v) * _pow2(-e)[..., None]
    a = v.abs()
    # to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; halfway to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(v).to(torch.uint8)).view(n, nope // 8, 2, 2, 2)  # p / 2, p % 2, h
    packed = (code[:, :, :, 0] + 16 * code[:, :, :, 1]).transpose(2, 3).reshape(n, nope // 2)
    scale = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    parts = [packed, x[:, nope:].contiguous().view(torch.uint8).view(n, 2 * pe), scale]
    used = nope // 2 + 2 * pe + nope // GROUP
    parts.append(torch.zeros(n, _row_bytes(nope, pe) - used, dtype=torch.uint8, device=x.device))
    return torch.cat(parts, 1)


def _decode(raw, nope, pe):
    """Cache rows [..., row] -> their values in fp32 [..., d]."""
    lead = raw.shape[:-1]
    b = raw[..., :nope // 2].reshape(*lead, nope // 8, 2, 2).transpose(-1, -2)  # p / 2, h
    code = torch.stack([b & 15, b >> 4], -2).reshape(*lead, nope).long()        # p / 2, p % 2, h
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=raw.device)[code]
    pes = raw[..., nope // 2:nope // 2 + 2 * pe].contiguous().view(torch.bfloat16).float()
    byte = raw[..., nope // 2 + 2 * pe:nope // 2 + 2 * pe + nope // GROUP].to(torch.int32)
    scale = torch.where(byte == 255, torch.full_like(byte, math.nan, dtype=torch.float32), _pow2(byte.clamp(1, 254) - 127))
    return torch.cat([value * scale.repeat_interleave(GROUP, -1), pes], -1)


# ---------------------------------------------------------------- inputs

def _freqs(pe, theta, factor, original=4096, fast=32.0, slow=1.0):
    """Radians a position of each pair, fp64 on the host, and the amplitude: theta^(-2i/pe), of
    which pairs that turn less than `slow` times within the original context are slowed down by
    `factor`, those that turn more than `fast` times are kept, and between a line joins the two."""
    i = torch.arange(pe // 2, dtype=torch.float64)
    f = theta ** (-2.0 * i / pe)
    if factor == 1.0:
        return f, 1.0
    pair = lambda turns: pe * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))  # noqa: E731
    low, high = max(0, math.floor(pair(fast))), min(pe - 1, math.ceil(pair(slow)))
    slowed = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f * (slowed / factor + 1 - slowed), 0.1 * math.log(factor) + 1


def _pages(st, case, g):
    """A pool in use: every sequence's pages, and a queue of the free ones that begins anywhere."""
    rows, page, width = case["rows"], case["page"], case["max_pages"]
    asked = torch.tensor(_asked(case), dtype=torch.int32, device="cuda")
    room = (width * page - asked.clamp(min=0)).clamp(min=0)
    # lengths over the whole range, the same ones whatever the seed, which gives them their order
    lens = (room * (torch.arange(rows, device="cuda") * 0.6180339887498949 % 1)).int().clamp(max=room)
    order = torch.randperm(rows, generator=g, device="cuda")
    new, lens = asked[order], lens[order]
    used = (lens + page - 1) // page
    total = int(used.sum())
    pool = total + case["free"]
    perm = torch.randperm(pool, generator=g, device="cuda").int()
    k = torch.arange(width, device="cuda")
    at = (torch.cumsum(used, 0) - used)[:, None] + k
    st["table"] = torch.where(k < used[:, None], perm[at.clamp(max=pool - 1)], -1).int()
    head = int(torch.randint(pool, (1,), generator=g, device="cuda"))
    queue = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    queue[(head + torch.arange(case["free"], device="cuda")) % pool] = perm[total:]
    st["queue"], st["new"] = queue, new
    st["state"] = torch.cat([lens, torch.tensor([head, case["free"]], dtype=torch.int32, device="cuda")])
    st["next"] = torch.empty_like(st["state"])
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "rope":
        kind = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["type"]]
        normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(kind)  # noqa: E731
        st["x"] = [normal(case["n"], case["nh"], case["d"])]
        if case["latent"]:
            st["x"].append(normal(case["n"], case["d"]))
        st["freqs"], st["amplitude"] = _freqs(case["pe"], 10000.0, case["factor"])
        st["freqs_there"] = st["freqs"].to("cuda")
        st["positions"] = torch.randint(0, 65536, (case["n"],), generator=g, device="cuda", dtype=torch.int32)
        return st
    if case["op"] == "pages":
        return _pages(st, case, g)
    if case["op"] == "slots":
        seqs, width = -(-case["rows"] // case["sq"]), -(-case["len"] // case["page"])
        st["table"] = torch.randperm(seqs * width + 1, generator=g, device="cuda")[:seqs * width].view(seqs, width).int()
        st["num_pages"] = seqs * width + 1
        # lengths from half to all of it; the indices, of any sequence's past, may lie behind a shorter one's end
        lens = case["len"] - case["len"] // 2 * torch.rand(seqs, generator=g, device="cuda")
        st["lens"] = lens.int().clamp(min=1)
        idx = torch.randint(0, case["len"], (case["rows"], case["topk"]), generator=g, device="cuda", dtype=torch.int32)
        pad = torch.rand(case["rows"], case["topk"], generator=g, device="cuda") < 0.05
        st["idx"] = torch.where(pad, torch.full_like(idx, -1), idx)
        return st
    nope, pe, page, d = case["nope"], case["pe"], case["page"], case["nope"] + case["pe"]

    def latents(n):
        """Vectors as a norm leaves them: unit size, with a few large channels."""
        x = torch.randn(n, d, generator=g, device="cuda")
        gain = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
        return (x * gain / gain.square().mean().sqrt()).to(torch.bfloat16)

    def pool(pages):
        return _encode(latents(pages * page), nope, pe).view(pages, page, -1)

    if case["op"] == "cache":
        slots = torch.randperm(case["pages"] * page, generator=g, device="cuda")[:case["n"]]
        if case["n"] > page:  # whole pages in any order, tokens in order inside them
            order = torch.randperm(case["pages"], generator=g, device="cuda")[:-(-case["n"] // page)]
            slots = (order[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:case["n"]]
        st["slots"] = slots.to(torch.int32)
        st["cache"] = pool(case["pages"])
        if case["write"]:
            st["x"] = latents(case["n"])
        return st
    rows, nh = case["rows"], case["nh"]
    st["q"] = torch.randn(rows, nh, d, generator=g, device="cuda").to(torch.bfloat16)
    st["scale"] = 1.0 / math.sqrt(d)
    if not case["picked"]:
        lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        st["lens"] = lens[torch.randperm(rows, generator=g, device="cuda")]
        width = max(1, -(-case["hi"] // page))
        pages = rows * width + 1
        st["table"] = torch.randperm(pages, generator=g, device="cuda")[:rows * width].view(rows, width).to(torch.int32)
        st["cache"] = pool(pages)
        return st
    idx = torch.randint(0, case["slots"], (rows, case["topk"]), generator=g, device="cuda", dtype=torch.int32)
    pad = torch.rand(rows, case["topk"], generator=g, device="cuda") < 0.05
    st["idx"] = torch.where(pad, torch.full_like(idx, -1), idx)
    st["cache"] = pool(-(-case["slots"] // page))
    return st


# ---------------------------------------------------------------- one pass

def _turned(x, cos, sin, pe, inter):
    """The last pe channels of x [n, heads, d] turned by the angles [n, 1, pe / 2], rounded once."""
    v = x.float()
    part = v[..., v.shape[-1] - pe:]
    a, b = (part[..., 0::2], part[..., 1::2]) if inter else (part[..., :pe // 2], part[..., pe // 2:])
    c, d = a * cos - b * sin, b * cos + a * sin
    part = torch.stack([c, d], -1).flatten(-2) if inter else torch.cat([c, d], -1)
    return torch.cat([v[..., :v.shape[-1] - pe], part], -1).to(x.dtype)


def _plain_rope(st):
    case = st["case"]
    angle = st["positions"].double()[:, None, None] * st["freqs_there"]
    cos, sin = (torch.cos(angle) * st["amplitude"]).float(), (torch.sin(angle) * st["amplitude"]).float()
    sin = -sin if case["back"] else sin
    first = _turned(st["x"][0], cos, sin, case["pe"], case["inter"])
    if not case["latent"]:
        return [first]
    return [first, _turned(st["x"][1][:, None], cos, sin, case["pe"], case["inter"])[:, 0]]


def _plain_pages(st):
    case, new, table, queue = st["case"], st["new"].long(), st["table"], st["queue"]
    page, width, pool, room, rows = case["page"], case["max_pages"], len(queue), _room(case), case["rows"]
    lens, head, count = st["state"][:rows].long(), st["state"][rows].long(), st["state"][rows + 1].long()
    asked = new.clamp(min=0)
    used = (lens + page - 1) // page
    fits = (asked > 0) & (lens + asked <= width * page)
    need = torch.where(fits, (lens + asked + page - 1) // page - used, 0)
    upto, pages_upto = torch.cumsum(asked, 0), torch.cumsum(need, 0)
    given = fits & ((need == 0) | (pages_upto <= count)) & (upto <= room)
    granted = torch.where(given, asked, 0)
    handed = torch.where(given, need, 0).sum()
    back = torch.where(new < 0, used, 0)
    # tokens
    t = torch.arange(room, device=new.device)
    row = torch.searchsorted(upto, t, right=True)
    real = row < rows
    row = row.clamp(max=rows - 1)
    ok = real & given[row]
    pos = lens[row] + t - (upto - asked)[row]
    k = torch.where(ok, pos // page, 0)
    fresh = (head + (pages_upto - need)[row] + k - used[row]) % pool
    where = torch.where(k < used[row], table[row, k].long(), queue[fresh].long())
    slots = torch.where(ok, where * page + pos % page, -1)
    first = ok & (pos % page == 0)
    # pages of sequences that ended go to the queue's end
    ended = torch.arange(width, device=new.device) < back[:, None]
    at = (head + count + (torch.cumsum(back, 0) - back)[:, None] + torch.arange(width, device=new.device)) % pool
    queue[at[ended]] = table[ended]
    table[row[first], k[first]] = where[first].int()
    st["next"][:rows] = torch.where(new < 0, 0, lens + granted)
    st["next"][rows] = (head + handed) % pool
    st["next"][rows + 1] = count - handed + back.sum()
    starts = torch.cat([torch.zeros_like(upto[:1]), upto]).clamp(max=room)
    return (slots.int(), torch.where(ok, pos, 0).int(), torch.where(real, row, -1).int(), starts.int(), granted.int(),
            st["next"], table, queue)


def _plain_slots(st):
    case, idx = st["case"], st["idx"]
    page, (seqs, width) = case["page"], st["table"].shape
    seq = torch.arange(case["rows"], device=idx.device)[:, None] // case["sq"]
    ok = (idx >= 0) & (idx < st["lens"][seq])
    token = torch.where(ok, idx, 0)
    return torch.where(ok, st["table"].view(-1)[seq * width + token // page] * page + token % page, -1).int()


def _attend(q, keys, valid, scale):
    """Softmax attention of q [rows, nh, d] over keys = values [rows, n, d]; a
    row with nothing to attend to gives zeros and a log-sum-exp of -inf."""
    keys = torch.where(valid[..., None], keys, torch.zeros_like(keys))
    s = torch.matmul(q.float(), keys.transpose(1, 2)) * scale
    s = torch.where(valid[:, None, :], s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, keys) / torch.where(total == 0, torch.ones_like(total), total)
    return o.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def _plain(st):
    case = st["case"]
    if case["op"] == "rope":
        return _plain_rope(st)
    if case["op"] == "pages":
        return _plain_pages(st)
    if case["op"] == "slots":
        return _plain_slots(st)
    nope, pe, cache = case["nope"], case["pe"], st["cache"]
    flat = cache.view(-1, cache.shape[-1])
    if case["op"] == "cache":
        slots = st["slots"].long()
        if case["write"]:
            flat[slots] = _encode(st["x"], nope, pe)
        return _decode(flat[slots], nope, pe).to(torch.bfloat16)
    if case["picked"]:
        slots = st["idx"].long()
        valid = slots >= 0
    else:
        page = cache.shape[1]
        t = torch.arange(max(1, case["hi"]), device=flat.device)
        valid = t[None, :] < st["lens"][:, None]
        slots = st["table"].long()[:, t // page] * page + t % page
    keys = _decode(flat[torch.where(valid, slots, torch.zeros_like(slots))], nope, pe)
    return _attend(st["q"], keys, valid, st["scale"])


def run(st):
    if not own:
        return _plain(st)
    import partial_inverse_rope_gb300 as ir
    case = st["case"]
    if case["op"] == "rope":
        return ir.rope_apply(st["x"], st["freqs"], st["positions"], amplitude=st["amplitude"], interleaved=case["inter"],
                             inverse=case["back"])
    if case["op"] == "pages":
        got = ir.kv_pages_advance(st["state"], st["table"], st["queue"], st["new"], case["page"], _room(case),
                                  state_out=st["next"])
        return (*got, st["next"], st["table"], st["queue"])
    if case["op"] == "slots":
        return ir.kv_idx_local_to_slots(st["idx"], st["table"], st["lens"], case["page"], st["num_pages"], case["sq"])
    nope, pe = case["nope"], case["pe"]
    if case["op"] == "cache":
        if case["write"]:
            ir.kv_latent_write(st["cache"], st["x"], st["slots"], nope, pe)
        return ir.kv_latent_read(st["cache"], st["slots"], nope, pe)
    if case["picked"]:
        return ir.latent_attn_sparse(st["q"], st["cache"], st["idx"], nope, pe, st["scale"])
    return ir.latent_attn_decode(st["q"], st["cache"], st["table"], st["lens"], nope, pe, st["scale"])


# ---------------------------------------------------------------- in 64 bits

def _exact_values(raw, nope, pe):
    """The values that cache rows stand for, in fp64, from the codes' bits."""
    words = raw[..., :nope // 2].contiguous().view(torch.int32).long()[..., None]
    c = torch.arange(8, device=raw.device)
    code = ((words >> (16 * (c % 2) + 4 * (c // 2))) & 15).flatten(-2)
    field, frac = (code >> 1) & 3, (code & 1).double() / 2
    size = torch.where(field == 0, frac, (1 + frac) * torch.exp2((field - 1).double()))
    value = torch.where(code >= 8, -size, size)
    byte = raw[..., nope // 2 + 2 * pe:nope // 2 + 2 * pe + nope // GROUP].long()
    scale = torch.exp2((byte - 127).double())
    scale = torch.where(byte == 255, torch.full_like(scale, math.nan), scale)
    halves = raw[..., nope // 2:nope // 2 + 2 * pe].contiguous().view(torch.bfloat16)
    return torch.cat([value * scale[..., torch.arange(nope, device=raw.device) // GROUP], halves.double()], -1)


def _exact_kept(x, nope):
    """What a vector reads as after it was written, in fp64."""
    v = x.double()
    for g0 in range(0, nope, GROUP):
        part = v[:, g0:g0 + GROUP]
        mant, exp = torch.frexp(part.abs().amax(-1, keepdim=True) / 6)
        step = torch.exp2(torch.where(mant == 0.5, exp - 1, exp).clamp(E_MIN, E_MAX).double())
        y = (part / step).abs()
        ulp = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=0).double() - 1)
        kept = (torch.round(y / ulp) * ulp).clamp(max=6) * step
        v[:, g0:g0 + GROUP] = torch.where(part < 0, -kept, kept)
    return v


def _exact_rope(st):
    case, out = st["case"], []
    angle = st["positions"].double()[:, None] * st["freqs_there"]
    turn = torch.polar(torch.full_like(angle, st["amplitude"]), -angle if case["back"] else angle)
    for x in st["x"]:
        v = x.double().view(case["n"], -1, case["d"])
        part = v[..., case["d"] - case["pe"]:]
        pairs = part.unflatten(-1, (-1, 2)) if case["inter"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
        v[..., case["d"] - case["pe"]:] = (pairs if case["inter"] else pairs.transpose(-1, -2)).flatten(-2)
        out.append(v.view(x.shape))
    return out


def _exact_pages(st):
    """One sequence after the other, as the definition says."""
    case, table, queue, state = st["case"], st["table"].tolist(), st["queue"].tolist(), st["state"].tolist()
    page, pool, room, rows = case["page"], len(queue), _room(case), case["rows"]
    head, count = state[rows:]
    slots, positions, row_of, starts, granted, lens = [], [], [], [0], [], []
    handed = asked_pages = 0
    tail = head + count
    back = []
    for r, n in enumerate(st["new"].tolist()):
        length = state[r]
        used = -(-length // page)
        if n < 0:
            back += table[r][:used]
            lens.append(0)
            granted.append(0)
            starts.append(starts[-1])
            continue
        need = -(-(length + n) // page) - used
        if length + n > case["max_pages"] * page:
            ok, need = False, 0
        else:
            asked_pages += need
            ok = n > 0 and (need == 0 or asked_pages <= count) and starts[-1] + n <= room
        if ok:
            table[r][used:used + need] = [queue[(head + handed + i) % pool] for i in range(need)]
            handed += need
        for t in range(length, length + n):
            slots.append(table[r][t // page] * page + t % page if ok else -1)
            positions.append(t if ok else 0)
            row_of.append(r)
        lens.append(length + (n if ok else 0))
        granted.append(n if ok else 0)
        starts.append(starts[-1] + n)
    for i, p in enumerate(back):
        queue[(tail + i) % pool] = p
    pad = room - len(slots)
    state = lens + [(head + handed) % pool, count - handed + len(back)]
    out = (slots + [-1] * pad, positions + [0] * pad, row_of + [-1] * pad, starts, granted, state, table, queue)
    return tuple(torch.tensor(v, dtype=torch.int32) for v in out)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "pages":
        return _exact_pages(st)
    if case["op"] == "slots":
        out = torch.full_like(st["idx"], -1)
        for s in range(len(st["lens"])):  # a sequence's slots in the order of its tokens
            t = torch.arange(int(st["lens"][s]), device=out.device)
            slot = (st["table"][s].repeat_interleave(case["page"])[t] * case["page"] + t % case["page"]).int()
            part = st["idx"][s * case["sq"]:(s + 1) * case["sq"]]
            ok = (part >= 0) & (part < len(slot))
            out[s * case["sq"]:(s + 1) * case["sq"]][ok] = slot[part[ok].long()]
        return out
    nope, pe, cache = case["nope"], case["pe"], st["cache"]
    flat = cache.view(-1, cache.shape[-1])
    if case["op"] == "cache":
        return _exact_kept(st["x"], nope) if case["write"] else _exact_values(flat[st["slots"].long()], nope, pe)
    outs, lses = [], []
    for r in range(case["rows"]):
        if case["picked"]:
            slots = st["idx"][r].long()
            slots = slots[slots >= 0]
        else:
            t = torch.arange(int(st["lens"][r]), device=flat.device)
            slots = st["table"][r].long()[t // cache.shape[1]] * cache.shape[1] + t % cache.shape[1]
        k = _exact_values(flat[slots], nope, pe)
        s = st["q"][r].double() @ k.T * st["scale"]
        lse = torch.logsumexp(s, -1)
        lses.append(lse)
        outs.append(torch.exp(s - lse[:, None]) @ k if len(slots) else torch.zeros_like(st["q"][r], dtype=torch.float64))
    return torch.stack(outs), torch.stack(lses)
