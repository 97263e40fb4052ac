"""Measured cases of the latent-cache operators: one serving step's parts over
a paged cache that holds one latent vector a token, which serves as key and as
value of every head.

* ``append``: new tokens' vectors are written into the cache (quantised where
  it holds 8-bit rows) and read back through their slots.
* ``read``: rows of a cache are read back by slot, as bf16.
* ``decode``: attention of one new token a sequence over its pages.
* ``sparse``: attention of query rows over the cache rows that an index table
  selects (the flat-global table that ``kv_idx_local_to_global`` makes).

``own`` chooses between elementary torch operations and the package's kernels.

A cache is a pool of pages. bf16 rows are ``d = nope + pe`` values; 8-bit rows
are ``nope`` e4m3 codes, ``pe`` bf16 values, one power-of-two scale byte
(biased by 127) for each 64 codes, and padding to 16 bytes.
"""

import math

import torch

own = False

GROUP = 64          # channels that share a scale
E_MIN, E_MAX = -120, 119


def listed():
    base = {"nope": 448, "pe": 64}
    return [
        # one decoding step of 64 sequences puts one token each into the cache
        {"name": "append_64_e4m3", "op": "append", "fmt": "e4m3", "n": 64, "pages": 2048, "page": 64, **base},
        # a prompt shard of 16384 tokens
        {"name": "append_16384_e4m3", "op": "append", "fmt": "e4m3", "n": 16384, "pages": 2048, "page": 64, **base},
        # a ragged prompt chunk into an unquantised cache
        {"name": "append_4097_bf16", "op": "append", "fmt": "bf16", "n": 4097, "pages": 2048, "page": 64, **base},
        # a short shared prefix
        {"name": "read_777_e4m3", "op": "read", "fmt": "e4m3", "n": 777, "pages": 2048, "page": 64, **base},
        # the whole of a 64K context, for a prompt that continues it
        {"name": "read_65536_e4m3", "op": "read", "fmt": "e4m3", "n": 65536, "pages": 2048, "page": 64, **base},
        # one user, a short conversation: latency
        {"name": "decode_1x200_bf16", "op": "decode", "fmt": "bf16", "rows": 1, "nh": 64, "lo": 200, "hi": 200, "page": 64, **base},
        # one user at the end of a 64K context: one row split over the whole card
        {"name": "decode_1x65536_e4m3", "op": "decode", "fmt": "e4m3", "rows": 1, "nh": 64, "lo": 65536, "hi": 65536, "page": 64, **base},
        # an ordinary serving batch, ragged
        {"name": "decode_32_ragged_bf16", "op": "decode", "fmt": "bf16", "rows": 32, "nh": 64, "lo": 1, "hi": 16384, "page": 64, **base},
        # a large batch over 8-bit rows
        {"name": "decode_96_ragged_e4m3", "op": "decode", "fmt": "e4m3", "rows": 96, "nh": 64, "lo": 4000, "hi": 20000, "page": 64, **base},
        # 128 heads, small pages
        {"name": "decode_24_nh128_bf16", "op": "decode", "fmt": "bf16", "rows": 24, "nh": 128, "lo": 2000, "hi": 16384, "page": 16, **base},
        # a decoding batch of 64 rows with 2048 selected rows each
        {"name": "sparse_64x2048_e4m3", "op": "sparse", "fmt": "e4m3", "rows": 64, "nh": 64, "topk": 2048, "slots": 65536, "page": 64, **base},
        # a prompt chunk, every row with its own selection
        {"name": "sparse_2048x2048_bf16", "op": "sparse", "fmt": "bf16", "rows": 2048, "nh": 64, "topk": 2048, "slots": 65536, "page": 64, **base},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "sparse"])
    nope, pe = rng.choice([(448, 64), (448, 64), (96, 32), (64, 64), (480, 32), (48, 16)])
    case = {"op": op, "fmt": rng.choice(["bf16", "e4m3"]), "nope": nope, "pe": pe,
            "page": rng.choice([1, 16, 48, 64, 64, 128])}
    if op in ("append", "read"):
        n = _spread(rng, 1, 65536 if op == "read" else 16384)
        return {**case, "n": n, "pages": -(-max(4 * n, 4096) // case["page"])}
    case["nh"] = rng.choice([1, 3, 16, 48, 64, 64, 96, 128])
    if op == "decode":
        rows = _spread(rng, 1, 128)
        hi = _spread(rng, 1, min(65536, 1 << 20) // max(1, rows // 16))
        return {**case, "rows": rows, "lo": rng.randint(0, hi), "hi": hi}
    rows = _spread(rng, 1, 1024)
    return {**case, "rows": rows, "topk": _spread(rng, 1, 2048), "slots": _spread(rng, 2048, 65536)}


def _row_bytes(case):
    if case["fmt"] == "bf16":
        return 2 * (case["nope"] + case["pe"])
    return -(-(case["nope"] + 2 * case["pe"] + -(-case["nope"] // GROUP)) // 16) * 16


def _lens(case):
    """Lengths from lo to hi in even steps: the same total whatever the seed."""
    r = case["rows"]
    return [case["hi"] if r == 1 else case["lo"] + (case["hi"] - case["lo"]) * i // (r - 1) for i in range(r)]


def work(case):
    d, rb = case["nope"] + case["pe"], _row_bytes(case)
    if case["op"] == "append":
        # the vectors in, the cache rows out, and the read back: rows in, vectors out
        return {"bytes": case["n"] * (2 * d + 2 * rb + 2 * d + 8), "flops": 0}
    if case["op"] == "read":
        return {"bytes": case["n"] * (rb + 2 * d + 4), "flops": 0}
    rows, nh = case["rows"], case["nh"]
    io = rows * nh * (4 * d + 4)  # queries in, outputs and log-sum-exp out
    if case["op"] == "decode":
        tokens = sum(_lens(case))
        table = 4 * sum(-(-n // case["page"]) for n in _lens(case))
        return {"bytes": tokens * rb + io + table + 4 * rows, "flops": 4 * tokens * nh * d}
    picked = rows * case["topk"]
    return {"bytes": min(picked, case["slots"]) * rb + io + 4 * picked, "flops": 4 * picked * nh * d}


# ---------------------------------------------------------------- the cache's rows

def _pow2(e):
    """2^e for whole e from -126 to 127, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x, nope, pe, fmt):
    """bf16 vectors [n, d] -> cache rows (bf16 [n, d] or uint8 [n, row bytes])."""
    if fmt == "bf16":
        return x.clone()
    n = x.shape[0]
    groups = -(-nope // GROUP)
    v = torch.zeros(n, groups * GROUP, device=x.device)
    v[:, :nope] = x[:, :nope].float()
    v = v.view(n, groups, GROUP)
    mant, exp = torch.frexp(v.abs().amax(-1))
    e = torch.where(mant <= 0.875, exp - 9, exp - 8).clamp(E_MIN, E_MAX)  # the least e with amax <= 448 * 2^e
    bad = ~torch.isfinite(v).all(-1)
    e = torch.where(bad, torch.zeros_like(e), e)
    v = torch.where(bad[..., None], torch.zeros_like(v), v)
    codes = (v * _pow2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    parts = [codes.view(n, -1)[:, :nope], x[:, nope:].contiguous().view(torch.uint8), scale]
    used = sum(p.shape[1] for p in parts)
    parts.append(torch.zeros(n, -(-used // 16) * 16 - used, dtype=torch.uint8, device=x.device))
    return torch.cat(parts, 1)


def _decode(raw, nope, pe, fmt):
    """Cache rows [..., row] -> their values in fp32 [..., d]."""
    if fmt == "bf16":
        return raw.float()
    codes = raw[..., :nope].contiguous().view(torch.float8_e4m3fn).float()
    pes = raw[..., nope:nope + 2 * pe].contiguous().view(torch.bfloat16).float()
    byte = raw[..., nope + 2 * pe:nope + 2 * pe + -(-nope // GROUP)].to(torch.int32)
    scale = torch.where(byte == 255, torch.full_like(byte, math.nan, dtype=torch.float32), _pow2(byte.clamp(1, 254) - 127))
    return torch.cat([codes * scale.repeat_interleave(GROUP, -1)[..., :nope], pes], -1)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nope, pe, page, d = case["nope"], case["pe"], case["page"], case["nope"] + case["pe"]

    def latents(n):
        """Vectors as a norm leaves them: unit size, with a few large channels."""
        x = torch.randn(n, d, generator=g, device="cuda")
        gain = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
        return (x * gain / gain.square().mean().sqrt()).to(torch.bfloat16)

    def pool(pages):
        return _encode(latents(pages * page), nope, pe, case["fmt"]).view(pages, page, -1)

    st = {"case": case, "nope": nope, "pe": pe}
    if case["op"] in ("append", "read"):
        slots = torch.randperm(case["pages"] * page, generator=g, device="cuda")[:case["n"]]
        if case["n"] > page:  # whole pages in any order, tokens in order inside them
            order = torch.randperm(case["pages"], generator=g, device="cuda")[:-(-case["n"] // page)]
            slots = (order[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:case["n"]]
        st["slots"] = slots.to(torch.int32)
        st["cache"] = pool(case["pages"])
        if case["op"] == "append":
            st["x"] = latents(case["n"])
        return st
    rows, nh = case["rows"], case["nh"]
    st["q"] = torch.randn(rows, nh, d, generator=g, device="cuda").to(torch.bfloat16)
    st["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "decode":
        lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        st["lens"] = lens[torch.randperm(rows, generator=g, device="cuda")]
        width = max(1, -(-case["hi"] // page))
        pages = rows * width + 1
        order = torch.randperm(pages, generator=g, device="cuda")[:rows * width].view(rows, width)
        st["table"] = order.to(torch.int32)
        st["cache"] = pool(pages)
        return st
    pages = -(-case["slots"] // page)
    idx = torch.randint(0, case["slots"], (rows, case["topk"]), generator=g, device="cuda", dtype=torch.int32)
    pad = torch.rand(rows, case["topk"], generator=g, device="cuda") < 0.05
    st["idx"] = torch.where(pad, torch.full_like(idx, -1), idx)
    st["cache"] = pool(pages)
    return st


# ---------------------------------------------------------------- one pass

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
    case, nope, pe = st["case"], st["nope"], st["pe"]
    cache, fmt = st["cache"], case["fmt"]
    flat = cache.view(-1, cache.shape[-1])
    if case["op"] in ("append", "read"):
        slots = st["slots"].long()
        if case["op"] == "append":
            flat[slots] = _encode(st["x"], nope, pe, fmt)
        return _decode(flat[slots], nope, pe, fmt).to(torch.bfloat16)
    if case["op"] == "decode":
        page = cache.shape[1]
        t = torch.arange(max(1, case["hi"]), device=flat.device)
        valid = t[None, :] < st["lens"][:, None]
        slots = st["table"].long()[:, t // page] * page + t % page
    else:
        slots = st["idx"].long()
        valid = slots >= 0
    keys = _decode(flat[torch.where(valid, slots, torch.zeros_like(slots))], nope, pe, fmt)
    return _attend(st["q"], keys, valid, st["scale"])


def run(st):
    if not own:
        return _plain(st)
    import partial_inverse_rope_gb300 as ir
    op, nope, pe = st["case"]["op"], st["nope"], st["pe"]
    if op == "append":
        ir.kv_latent_write(st["cache"], st["x"], st["slots"], nope, pe)
        return ir.kv_latent_read(st["cache"], st["slots"], nope, pe)
    if op == "read":
        return ir.kv_latent_read(st["cache"], st["slots"], nope, pe)
    if op == "decode":
        return ir.latent_attn_decode(st["q"], st["cache"], st["table"], st["lens"], nope, pe, st["scale"])
    return ir.latent_attn_sparse(st["q"], st["cache"], st["idx"], nope, pe, st["scale"])


# ---------------------------------------------------------------- in 64 bits

def _exact_values(raw, nope, pe, fmt):
    """The values that cache rows stand for, in fp64, from the codes' bits."""
    if fmt == "bf16":
        return raw.double()
    c = raw[..., :nope].long()
    field, frac = (c >> 3) & 15, (c & 7).double() / 8
    size = torch.where(field == 0, torch.ldexp(frac, torch.tensor(-6.0, device=c.device)),
                       (1 + frac) * torch.exp2((field - 7).double()))
    value = torch.where(c >= 128, -size, size)
    byte = raw[..., nope + 2 * pe:nope + 2 * pe + -(-nope // GROUP)].long()
    scale = torch.exp2((byte - 127).double())
    scale = torch.where(byte == 255, torch.full_like(scale, math.nan), scale)
    group = torch.arange(nope, device=c.device) // GROUP
    halves = raw[..., nope:nope + 2 * pe].contiguous().view(torch.bfloat16)
    return torch.cat([value * scale[..., group], halves.double()], -1)


def _exact_kept(x, nope, fmt):
    """What a vector reads as after it was written, in fp64."""
    v = x.double()
    if fmt == "bf16":
        return v
    for g0 in range(0, nope, GROUP):
        part = v[:, g0:min(nope, g0 + GROUP)]
        ratio = part.abs().amax(-1, keepdim=True) / 448
        mant, exp = torch.frexp(ratio)
        step = torch.exp2(torch.where(mant == 0.5, exp - 1, exp).clamp(E_MIN, E_MAX).double())
        y = (part / step).abs()
        ulp = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
        kept = (torch.round(y / ulp) * ulp).clamp(max=448) * step
        v[:, g0:min(nope, g0 + GROUP)] = torch.where(part < 0, -kept, kept)
    return v


def exact(case, seed):
    st = prepare(case, seed)
    nope, pe, fmt = st["nope"], st["pe"], case["fmt"]
    cache = st["cache"]
    flat = cache.view(-1, cache.shape[-1])
    if case["op"] == "append":
        return _exact_kept(st["x"], nope, fmt)
    if case["op"] == "read":
        return _exact_values(flat[st["slots"].long()], nope, pe, fmt)
    outs, lses = [], []
    lens = st["lens"].tolist() if case["op"] == "decode" else [case["topk"]] * case["rows"]
    for r, n in enumerate(lens):
        if case["op"] == "decode":
            page = cache.shape[1]
            t = torch.arange(n, device=flat.device)
            slots = st["table"][r].long()[t // page] * page + t % page
        else:
            slots = st["idx"][r].long()
            slots = slots[slots >= 0]
        k = _exact_values(flat[slots], nope, pe, fmt)
        s = st["q"][r].double() @ k.T * st["scale"]
        lse = torch.logsumexp(s, -1)
        lses.append(lse)
        outs.append(torch.exp(s - lse[:, None]) @ k if len(slots) else torch.zeros_like(st["q"][r], dtype=torch.float64))
    return torch.stack(outs), torch.stack(lses)
