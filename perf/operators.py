"""The paged 4-bit key/value cache's operators: cases, inputs, plain forms and exact values.

Four operations of a serving step around the draft sampler and its verification:

  append   quantise the step's new keys and values into their requests' pages (4-bit E2M1 codes, one E4M3 scale for
           each 16 of them, one FP32 scale for each head), and read back the values that the cache now stands for
  attend   attention of each request's newest rows over its pages: single tokens, the P + 1 rows of a verification,
           chunks of a prompt; grouped heads, causal, with or without a sliding window
  branch   one round of branching drafts: drop the last round's branches, fork every request, grow the branches'
           page tables (lowest free pages first, a shared last page copied on write), copy the pages' data
  compact  move the live pages into the lowest page ids, renumber the page tables, copy the moved pages' data

Layout of a page: one record for each key/value head, `page * (dim + dim / 8)` bytes: key codes [page, dim / 2], value
codes [page, dim / 2], key scales [page, dim / 16], value scales [page, dim / 16]; byte j of a row of codes holds element
2 j in its low four bits and 2 j + 1 in its high four.  Rows of request i are row_start[i] .. row_start[i + 1] - 1; they
are the last rows of its lens[i] cached ones.
"""
import random

import torch

own = False

LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of E2M1
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------

def _append(name, requests, rows, past, page, kv_heads, dim, dtype="bf16", scaled=False):
    return dict(name=name, op="append", requests=requests, rows_lo=rows[0], rows_hi=rows[1], past=past, page=page,
                kv_heads=kv_heads, dim=dim, dtype=dtype, scaled=scaled)


def _attend(name, requests, rows, lens, page, kv_heads, group, dim, dtype="bf16", window=0, scaled=False):
    return dict(name=name, op="attend", requests=requests, rows_lo=rows[0], rows_hi=rows[1], len_lo=lens[0],
                len_hi=lens[1], page=page, kv_heads=kv_heads, group=group, dim=dim, dtype=dtype, window=window,
                scaled=scaled)


def _branch(name, requests, branches, rows, lens, page, kv_heads, dim, layers):
    return dict(name=name, op="branch", requests=requests, branches=branches, rows=rows, len_lo=lens[0],
                len_hi=lens[1], page=page, kv_heads=kv_heads, dim=dim, layers=layers)


def _compact(name, slots, lens, page, kv_heads, dim, layers, live):
    return dict(name=name, op="compact", slots=slots, len_lo=lens[0], len_hi=lens[1], page=page, kv_heads=kv_heads,
                dim=dim, layers=layers, live=live)


def listed():
    return [
        # A verification of 16 requests with 5 drafts each: 6 new rows a request.  Latency counts.
        _append("append verify 16x6", 16, (6, 6), 4000, 64, 8, 128),
        # Prompts of mixed lengths entering the cache, with a calibrated scale for each head.
        _append("append prompts", 12, (1, 4001), 1000, 32, 8, 128, "bf16", True),
        # One request, one token, a short context: the smallest attention call.
        _attend("attend 1x1 2k", 1, (1, 1), (2048, 2048), 64, 8, 8, 128),
        # Decoding a full batch of requests of mixed lengths, one token each.
        _attend("attend 64x1 16k", 64, (1, 1), (4096, 16384), 64, 8, 8, 128),
        # A few very long contexts, one token each: few rows, the work is along the cache.
        _attend("attend 3x1 128k", 3, (1, 1), (100001, 131072), 128, 8, 4, 128, "f16"),
        # The verification of 5 drafts (6 rows) for a batch of requests.
        _attend("attend verify 48x6 8k", 48, (6, 6), (1024, 8192), 64, 8, 8, 128),
        # A chunk of a long prompt: 2048 rows that attend to what is cached before them and to themselves.
        _attend("attend chunk 2048 of 16k", 1, (2048, 2048), (16384, 16384), 64, 8, 8, 128),
        # A mixed step of odd sizes: idle requests, single tokens and short prompts together; small heads, an odd
        # group, small pages, a sliding window, head scales.
        _attend("attend mixed odd", 23, (0, 133), (0, 3001), 16, 5, 5, 64, "f16", 1000, True),
        # Branching drafts of a small batch: 4 branches of 8 requests.
        _branch("branch 8x4", 8, 4, 6, (500, 2000), 64, 8, 128, 1),
        # The same for a large batch over the cache's layers.
        _branch("branch 128x4, 8 layers", 128, 4, 6, (1000, 8000), 64, 8, 128, 8),
        # Defragmenting a small pool after half of its requests have ended.
        _compact("compact small", 16, (100, 900), 16, 2, 64, 1, 0.5),
        # Defragmenting a large pool, several layers.
        _compact("compact large, 4 layers", 256, (1000, 5000), 64, 8, 128, 4, 0.6),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, odd above 16."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return min(hi, v | 1) if v > 16 else v


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "attend", "branch", "compact"))
    page = rng.choice((16, 32, 64, 128))
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    scaled = rng.random() < 0.5
    if op == "append":
        requests = _log(rng, 1, 200)
        rows = _log(rng, 1, max(2, 40000 // requests))
        c = _append("", requests, (rng.choice((1, rows)) if rows < 40 else 1, rows), _log(rng, 1, 4001), page,
                    kv_heads, dim, dtype, scaled)
    elif op == "attend":
        group = rng.choice((1, 2, 4, 5, 7, 8, 16))
        window = rng.choice((0, 0, 0, _log(rng, 17, 5001)))
        kind = rng.choice(("one", "verify", "chunk"))
        if kind == "one":
            requests = _log(rng, 1, 151)
            lens, rows = _log(rng, 1, min(131071, 400000 // requests)), (1, 1)
        elif kind == "verify":
            requests = _log(rng, 1, 101)
            lens, rows = _log(rng, 8, min(65535, 250000 // requests)), (rng.choice((0, 1, 2)), rng.choice((2, 4, 6, 8)))
        else:
            requests = _log(rng, 1, 9)
            hi = _log(rng, 17, 2001)
            lens = _log(rng, hi, max(hi, 16001 // requests))
            rows = (rng.choice((1, hi)), hi)
        c = _attend("", requests, rows, (rng.choice((0, lens // 2, lens)), lens), page, kv_heads, group, dim, dtype,
                    window, scaled)
    elif op == "branch":
        requests = _log(rng, 1, 151)
        layers = rng.choice((1, 2, 4, 8))
        lens = _log(rng, 17, min(8001, 4000000 // (requests * layers)))
        c = _branch("", requests, rng.choice((2, 3, 4)), rng.choice((1, 2, 6, 8)), (lens // 3, lens), page, kv_heads,
                    dim, layers)
    else:
        slots = _log(rng, 2, 251)
        layers = rng.choice((1, 2, 4))
        lens = _log(rng, 17, min(8001, 3000000 // (slots * layers)))
        c = _compact("", slots, (lens // 4, lens), page, kv_heads, dim, layers, rng.choice((0.3, 0.5, 0.8)))
    del c["name"]
    return c


def _record(c):
    """Bytes of one head's record of a page."""
    return c["page"] * (c["dim"] + c["dim"] // 8)


def _pages(n, page):
    return -(-n // page)


def _shape(c):
    """Rows and lengths of a case's requests (of its slots, for compact), and which slots live: the same whatever the
    seed, so that outputs of two seeds have one shape."""
    rng = random.Random(",".join("%s=%s" % (k, c[k]) for k in sorted(c) if k != "name"))
    n = c["slots"] if c["op"] == "compact" else c["requests"]
    if c["op"] == "append":
        rows = [rng.randint(c["rows_lo"], c["rows_hi"]) for _ in range(n)]
        return rows, [rng.randint(0, c["past"]) + r for r in rows], None
    lens = [rng.randint(c["len_lo"], c["len_hi"]) for _ in range(n)]
    if c["op"] == "attend":
        rows = [rng.randint(c["rows_lo"], c["rows_hi"]) for _ in range(n)]
        if c["len_lo"]:  # else some requests have more rows than cached tokens: rows that see nothing
            rows = [min(r, t) for r, t in zip(rows, lens)]
        rows[-1] = max(rows[-1], 1)
        return rows, lens, None
    return None, lens, [rng.random() < c.get("live", 1) for _ in range(n)]


def work(case):
    c = case
    rows, lens, live = _shape(c)
    if c["op"] == "append":
        elems = sum(rows) * c["kv_heads"] * c["dim"] * 2
        # the values in, the codes and scales out; the same back for the read
        return {"bytes": elems * (2 + 9 / 16) * 2, "flops": elems * 4}
    if c["op"] == "attend":
        pairs = read = 0
        for n, t in zip(rows, lens):
            span = c["window"] or t
            first = max(0, t - n + 1 - span) if n else t
            read += t - first
            # row i of n sees positions up to t - n + i, at most `span` of them
            below = min(n, max(0, n - t))  # rows that see nothing
            upto = max(1, t - n + 1)  # what the first row that sees something sees
            count = n - below
            ramp = min(count, max(0, span - upto))  # rows that the window does not cut
            pairs += ramp * upto + ramp * (ramp - 1) // 2 + (count - ramp) * min(span, t)
        heads = c["kv_heads"] * c["group"]
        return {"bytes": sum(rows) * heads * c["dim"] * 4 + read * c["kv_heads"] * c["dim"] * 9 / 8,
                "flops": pairs * heads * c["dim"] * 4}
    page, page_bytes = c["page"], _record(c) * c["kv_heads"] * c["layers"]
    if c["op"] == "branch":
        copies = sum(t % page != 0 for t in lens) * (c["branches"] - 1)
        entries = sum(_pages(t + c["rows"], page) for t in lens) * c["branches"]
        return {"bytes": 2 * copies * page_bytes + entries * 4 * 4, "flops": 0}
    held = sum(_pages(t, page) for t, a in zip(lens, live) if a)
    total = sum(_pages(t, page) for t in lens) + 3
    # live pages above the first `held` ids, their ids being a random choice
    return {"bytes": 2 * held * (1 - held / total) * page_bytes + total * 4 * 4, "flops": 0}


# ---------------------------------------------------------------------------------------------------------------------
# The plain form of the cache: quantising, storing and reading, 32-bit arithmetic on torch operations
# ---------------------------------------------------------------------------------------------------------------------

def _quantise(x, g):
    """x [..., heads, dim] -> codes (uint8, one a value), scales (uint8 E4M3, one for 16); g: [heads] or None."""
    y = x.float()
    if g is not None:
        y = y / g[:, None]
    y = torch.where(torch.isnan(y), torch.zeros_like(y), y).reshape(*x.shape[:-1], -1, 16)
    top = y.abs().amax(-1) / 6.0
    scale = top.clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    a = y.abs() / s
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where(s > 0, code, torch.zeros_like(code)) + 8 * (y < 0)
    return code.to(torch.uint8).reshape(x.shape), scale.view(torch.uint8)


def _values(code, scale, g):
    """The FP32 values that codes and scales stand for."""
    lut = torch.tensor(LUT + tuple(-v for v in LUT), device=code.device)
    v = lut[code.int()].reshape(*code.shape[:-1], -1, 16) * scale.view(torch.float8_e4m3fn).float()[..., None]
    v = v.reshape(code.shape)
    return v if g is None else v * g[:, None]


def _sections(data, c):
    """The four sections of a pool's bytes [pages, heads * record] as views: key codes, value codes, key scales, value
    scales, each [pages, heads, page, bytes]."""
    p, d, h = c["page"], c["dim"], c["kv_heads"]
    r = data.reshape(data.shape[0], h, _record(c))
    half, eighth = p * d // 2, p * d // 16
    cut = lambda at, n: r[:, :, at:at + n].unflatten(2, (p, n // p))  # noqa: E731
    return cut(0, half), cut(half, half), cut(2 * half, eighth), cut(2 * half + eighth, eighth)


def _store(data, c, page_of, row_of, k, v, gk, gv):
    """Writes rows k, v [rows, heads, dim] to rows `row_of` of pages `page_of`; returns their codes and scales."""
    kc, vc, ks, vs = _sections(data, c)
    out = []
    for codes, scales, x, g in ((kc, ks, k, gk), (vc, vs, v, gv)):  # keys, then values
        code, scale = _quantise(x, g)
        codes[page_of, :, row_of] = code[..., 0::2] | (code[..., 1::2] << 4)
        scales[page_of, :, row_of] = scale
        out.append((code, scale))
    return out


def _cached(data, c, table, length, gk, gv):
    """The cached keys and values of table rows [n, pages] up to `length` tokens, FP32 [n, heads, length, dim]."""
    n = _pages(length, c["page"])
    got = []
    picked = _sections(data[table[:, :n].clamp(min=0).long()].flatten(0, 1), c)
    for codes, scales, g in ((picked[0], picked[2], gk), (picked[1], picked[3], gv)):  # keys, then values
        code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        x = _values(code, scales.contiguous(), None if g is None else g[:, None])
        got.append(x.unflatten(0, (table.shape[0], n)).transpose(1, 2).flatten(2, 3)[:, :, :length])
    return got


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(need, page_ids, width):
    """Page tables [slots, width] that take need[i] of the ids in order, -1 behind them."""
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = page_ids[at:at + n]
        at += n
    return table


def _rows(n, heads, dim, dtype, gen, spread):
    """Activations as a projection gives them: normal, with some channels several times larger than the others."""
    channel = torch.exp(spread * torch.randn(heads, dim, device="cuda", generator=gen))
    return (torch.randn(n, heads, dim, device="cuda", generator=gen) * channel).to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    if c["op"] in ("branch", "compact"):
        return _prepare_pages(c, gen, cpu)
    dtype, h, d, b = TYPES[c["dtype"]], c["kv_heads"], c["dim"], c["requests"]
    rows, lens, _ = _shape(c)
    need = [_pages(n, c["page"]) for n in lens]
    num_pages = sum(need) + 5
    ids = torch.randperm(num_pages, generator=cpu).int()
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    total = starts[-1]
    scales = [None, None]
    if c["scaled"]:  # as calibration leaves them: about the largest magnitude over what codes and scales reach
        scales = [torch.exp(0.5 * torch.randn(h, device="cuda", generator=gen)) * 0.02 for _ in range(2)]
    s = dict(c=c, row_start=_ints(starts), lens=_ints(lens), table=_tables(need, ids, max(1, max(need))).cuda(),
             gk=scales[0], gv=scales[1], total=total, most=max(rows), longest=max(lens),
             data=torch.randint(0, 256, (num_pages, h * _record(c)), dtype=torch.uint8, device="cuda", generator=gen))
    if c["op"] == "append":
        s["k"] = _rows(total, h, d, dtype, gen, 0.7)
        s["v"] = _rows(total, h, d, dtype, gen, 0.3)
        s["k_seen"], s["v_seen"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    else:
        for at in range(0, num_pages, 2048):  # a cache that an earlier step filled
            part = s["data"][at:at + 2048]
            n = part.shape[0] * c["page"]
            page_of = torch.arange(n, device="cuda") // c["page"]
            row_of = torch.arange(n, device="cuda") % c["page"]
            _store(part, c, page_of, row_of, _rows(n, h, d, dtype, gen, 0.4), _rows(n, h, d, dtype, gen, 0.3),
                   s["gk"], s["gv"])
        s["q"] = _rows(total, h * c["group"], d, dtype, gen, 0.4)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = d ** -0.5
    if own:
        from dspark_markov_draft_anchor_gb300 import binding
        s["cache"] = binding.Kv4Cache(s["data"], c["page"], h, d, k_scale=s["gk"], v_scale=s["gv"])
        s["batch"] = binding.Kv4Batch(s["row_start"], s["lens"], s["table"], total_rows=total, max_rows=s["most"])
        if c["op"] == "attend":
            size = binding.dspark_kv4_attention_workspace_bytes(s["cache"], s["batch"], h * c["group"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _prepare_pages(c, gen, cpu):
    h, page = c["kv_heads"], c["page"]
    _, lens, live = _shape(c)
    if c["op"] == "branch":
        b, k = c["requests"], c["branches"]
        slots = b * k
        most = max(lens) + c["rows"]
        lens = lens + [0] * (slots - b)
        spare = slots * (2 + _pages(c["rows"], page))
    else:
        most = max(lens)
        spare = sum(_pages(n, page) for n, a in zip(lens, live) if not a) + 3
        lens = [n if a else 0 for n, a in zip(lens, live)]
    need = [_pages(n, page) for n in lens]
    num_pages = sum(need) + spare
    ids = torch.randperm(num_pages, generator=cpu).int()
    table = _tables(need, ids, _pages(most, page) + 1)
    refs = torch.zeros(num_pages, dtype=torch.int32)
    refs[ids[:sum(need)].long()] = 1
    s = dict(c=c, refs=refs.cuda(), table=table.cuda(), lens=_ints(lens))
    s["data"] = torch.randint(0, 256, (c["layers"], num_pages, h * _record(c)), dtype=torch.uint8, device="cuda",
                              generator=gen)
    if c["op"] == "branch":
        order = list(range(b, slots)) + list(range(b))  # the branches first: the request then keeps its last page
        s["every"] = _ints(order)
        s["base"] = _ints([lens[i] for i in order])
        s["add"] = _ints([c["rows"]] * slots)
        s["src"] = _ints([i for i in range(b) for _ in range(k - 1)])
        s["dst"] = _ints(list(range(b, slots)))
        s["copy_src"], s["copy_dst"], s["granted"] = (_ints([0] * slots) for _ in range(3))
    else:
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["map"], s["move_src"], s["move_dst"] = (torch.empty_like(s["refs"]) for _ in range(3))
        s["count"] = _ints([0])
    if own:
        from dspark_markov_draft_anchor_gb300 import binding
        s["pool"] = binding.PagePool(s["refs"], s["table"], s["lens"], page)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "branch": _own_branch, "compact": _own_compact}[op](s)
    return {"append": _plain_append, "attend": _plain_attend, "branch": _plain_branch, "compact": _plain_compact}[op](s)


def _own_append(s):
    from dspark_markov_draft_anchor_gb300 import binding
    binding.dspark_kv4_append(s["cache"], s["batch"], s["k"], s["v"])
    binding.dspark_kv4_read(s["cache"], s["batch"], s["k_seen"], s["v_seen"])
    return s["k_seen"], s["v_seen"]


def _own_attend(s):
    from dspark_markov_draft_anchor_gb300 import binding
    binding.dspark_kv4_attention(s["cache"], s["batch"], s["q"], s["out"], s["scale"], s["workspace"],
                                 window=s["c"]["window"])
    return s["out"]


def _own_branch(s):
    from dspark_markov_draft_anchor_gb300 import binding
    binding.dspark_pages_trim(s["pool"], s["every"], s["base"])
    binding.dspark_pages_fork(s["pool"], s["src"], s["dst"])
    binding.dspark_pages_grow(s["pool"], s["every"], s["add"], s["copy_src"], s["copy_dst"], s["granted"])
    binding.dspark_pages_copy(s["data"], s["copy_src"], s["copy_dst"])
    return {k: s[k] for k in ("table", "refs", "lens", "copy_src", "copy_dst", "granted", "data")}


def _own_compact(s):
    from dspark_markov_draft_anchor_gb300 import binding
    binding.dspark_pages_compact(s["pool"], s["table_out"], s["refs_out"], s["map"], s["move_src"], s["move_dst"],
                                 s["count"])
    binding.dspark_pages_copy(s["data"], s["move_src"], s["move_dst"], count=s["count"])
    return {k: s[k] for k in ("table_out", "refs_out", "map", "move_src", "move_dst", "count", "data")}


def _owner(s):
    """For each row: its request, and its position in the request's cache."""
    start, total = s["row_start"].long(), s["total"]
    row = torch.arange(total, device="cuda")
    owner = torch.searchsorted(start[1:], row, right=True)
    return owner, row - start[owner + 1] + s["lens"].long()[owner]


def _plain_append(s):
    c = s["c"]
    owner, pos = _owner(s)
    page_of = s["table"].long()[owner, pos // c["page"]]
    (kc, ks), (vc, vs) = _store(s["data"], c, page_of, pos % c["page"], s["k"], s["v"], s["gk"], s["gv"])
    dtype = TYPES[c["dtype"]]
    return _values(kc, ks, s["gk"]).to(dtype), _values(vc, vs, s["gv"]).to(dtype)


def _plain_attend(s):
    c = s["c"]
    b, h, g, d = c["requests"], c["kv_heads"], c["group"], c["dim"]
    n, t, total = s["most"], s["longest"], s["total"]
    if n == 0 or t == 0:
        return torch.zeros_like(s["q"])
    start, lens = s["row_start"].long(), s["lens"].long()
    count = start[1:] - start[:-1]
    row = torch.arange(n, device="cuda")
    at = (start[:-1, None] + row).clamp(max=total - 1)
    q = s["q"][at].float().unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).reshape(b, h, n * g, d)
    k, v = _cached(s["data"], c, s["table"], t, s["gk"], s["gv"])
    score = (q @ k.transpose(2, 3)) * s["scale"]
    pos = (lens[:, None] - count[:, None] + row)[:, :, None]  # of each row, in its request
    key = torch.arange(t, device="cuda")
    seen = (key <= pos) & (key < lens[:, None, None]) & (row < count[:, None])[:, :, None]
    if c["window"]:
        seen &= key > pos - c["window"]
    score = score.unflatten(2, (n, g)).masked_fill_(~seen[:, None, :, None, :], -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)))
    low = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, (n, g)) / torch.where(low > 0, low, torch.ones_like(low))
    out = out.permute(0, 2, 1, 3, 4).reshape(b * n, h * g, d)
    owner, _ = _owner(s)
    return out[owner * n + torch.arange(total, device="cuda") - start[owner]].to(s["q"].dtype)


def _release(s, slots, old, new):
    """Drops the pages of `slots` from page number `new` up to `old`: their references and their table entries."""
    col = torch.arange(s["table"].shape[1], device="cuda")
    rows = s["table"][slots]
    gone = (col >= new[:, None]) & (col < old[:, None])
    s["refs"].index_add_(0, rows[gone].long(), torch.full((1,), -1, dtype=torch.int32, device="cuda").expand(int(gone.sum())))
    s["table"][slots] = rows.masked_fill(gone, -1)


def _copy(data, src, dst):
    keep = src >= 0
    data[:, dst[keep].long()] = data[:, src[keep].long()]


def _plain_branch(s):
    page = s["c"]["page"]
    up = lambda n: (n + page - 1) // page  # noqa: E731
    refs, table, lens = s["refs"], s["table"], s["lens"]
    # drop what the last round grew
    slots = s["every"].long()
    old, new = lens[slots], torch.minimum(lens[slots], s["base"])
    _release(s, slots, up(old), up(new))
    lens[slots] = new
    # fork
    src, dst = s["src"].long(), s["dst"].long()
    col = torch.arange(table.shape[1], device="cuda")
    rows = table[src].masked_fill(col >= up(lens[src])[:, None], -1)
    table[dst] = rows
    lens[dst] = lens[src]
    refs += torch.bincount(rows[rows >= 0].long(), minlength=refs.numel()).int()
    # grow: new pages, and a copy of a last page that others hold too
    cur, add = lens[slots], s["add"]
    have = up(cur)
    index = torch.arange(slots.numel(), device="cuda")
    part = (add > 0) & (cur % page != 0)
    last = table[slots, (have - 1).clamp(min=0).long()].long().clamp(min=0)
    holders = torch.bincount(last[part], minlength=refs.numel())
    final = torch.full_like(holders, -1).scatter_reduce(0, last[part], index[part], "amax")
    stays = (holders[last] == refs[last]) & (final[last] == index)
    copied = part & (refs[last] > 1) & ~stays
    fresh = up(cur + add) - have
    want = fresh + copied.int()
    end = want.cumsum(0)
    free = torch.nonzero(refs == 0).flatten()
    fits = (cur + add) <= page * table.shape[1]
    granted = ((end <= free.numel()) | (want == 0)) & fits
    first = (end - want).long()
    take = granted & copied
    mine = free[first.clamp(max=free.numel() - 1)]
    s["copy_src"].copy_(torch.where(take, last, torch.full_like(last, -1)))
    s["copy_dst"].copy_(torch.where(take, mine, torch.full_like(mine, -1)))
    s["granted"].copy_(granted)
    table[slots[take], (have - 1)[take].long()] = mine[take].int()
    refs.sub_(torch.bincount(last[take], minlength=refs.numel()).int())
    nth = col - have[:, None] + copied[:, None].int()
    adds = granted[:, None] & (col >= have[:, None]) & (col < (have + fresh)[:, None])
    ids = free[(first[:, None] + nth).clamp(min=0, max=free.numel() - 1)].int()
    table[slots] = torch.where(adds, ids, table[slots])
    refs[ids[adds].long()] = 1
    refs[mine[take]] = 1
    lens[slots] = torch.where(granted, cur + add, cur)
    _copy(s["data"], s["copy_src"], s["copy_dst"])
    return {k: s[k] for k in ("table", "refs", "lens", "copy_src", "copy_dst", "granted", "data")}


def _plain_compact(s):
    refs = s["refs"]
    live = refs > 0
    n = refs.numel()
    ids = torch.arange(n, device="cuda")
    total = live.sum()
    src = ids[live & (ids >= total)]
    dst = ids[~live & (ids < total)]
    m = src.numel()
    to = torch.where(live, ids, torch.full_like(ids, -1))
    to[src] = dst
    s["map"].copy_(to)
    for name, x in (("move_src", src), ("move_dst", dst)):
        s[name].fill_(-1)
        s[name][:m] = x.int()
    s["count"].fill_(m)
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()].int(), s["table"]))
    s["refs_out"].zero_()
    s["refs_out"][to[live]] = refs[live]
    _copy(s["data"], s["move_src"], s["move_dst"])
    return {k: s[k] for k in ("table_out", "refs_out", "map", "move_src", "move_dst", "count", "data")}


# ---------------------------------------------------------------------------------------------------------------------
# 64-bit values
# ---------------------------------------------------------------------------------------------------------------------

def _nibble64(n):
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    return torch.where((n & 8) != 0, -mag, mag)


def _e4m3_64(byte):
    e, m = (byte >> 3) & 15, (byte & 7).double() / 8
    mag = torch.where(e == 0, m * 2.0 ** -6, (1 + m) * torch.exp2((e - 7).double()))
    return torch.where((byte & 128) != 0, -mag, mag)


def _round64(x, bits, least):
    """x >= 0 to the nearest number of `bits` significant bits, ties to even, on a grid no finer than `least`."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=1e-300))) - (bits - 1)).clamp(min=least)
    return torch.round(x / step) * step


def _quantised64(x, g):
    y = x.double() if g is None else x.double() / g.double()[:, None]
    y = y.reshape(*x.shape[:-1], -1, 16)
    s = _round64((y.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0), 4, 2.0 ** -9).clamp(max=448.0)
    a = (y.abs() / s.clamp(min=1e-300)).clamp(max=6.0)
    v = torch.where(s > 0, _round64(a, 2, 0.5) * s, torch.zeros_like(y)) * torch.sign(y)
    v = v.reshape(x.shape)
    return v if g is None else v * g.double()[:, None]


def exact(case, seed):
    c = case
    if c["op"] in ("branch", "compact"):
        return None
    s = prepare(c, seed)
    if c["op"] == "append":
        return _quantised64(s["k"], s["gk"]), _quantised64(s["v"], s["gv"])
    h, g, d, page = c["kv_heads"], c["group"], c["dim"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens = s["row_start"].tolist(), s["lens"].tolist()
    half, eighth = page * d // 2, page * d // 16
    for i in range(c["requests"]):
        n, t = starts[i + 1] - starts[i], lens[i]
        if n == 0 or t == 0:
            continue
        pages = s["table"][i, :_pages(t, page)].long()
        pos = torch.arange(n, device="cuda") + t - n
        key = torch.arange(t, device="cuda")
        seen = key[None] <= pos[:, None]
        if c["window"]:
            seen = seen & (key[None] > pos[:, None] - c["window"])
        for j in range(h):
            rec = s["data"][pages, j * _record(c):(j + 1) * _record(c)].int()
            both = []
            for at, sc, w in ((0, 2 * half, s["gk"]), (half, 2 * half + eighth, s["gv"])):
                byte = rec[:, at:at + half].reshape(-1, d // 2)[:t]
                x = torch.empty(t, d, dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = _nibble64(byte & 15), _nibble64(byte >> 4)
                by = _e4m3_64(rec[:, sc:sc + eighth].reshape(-1, d // 16)[:t])
                x *= by.repeat_interleave(16, 1)
                both.append(x if w is None else x * w[j].double())
            k, v = both
            for m in range(g):
                q = s["q"][starts[i]:starts[i + 1], j * g + m].double()
                w = torch.where(seen, (q @ k.T) * s["scale"], torch.full((1, 1), -torch.inf, dtype=torch.float64, device="cuda"))
                w = torch.softmax(w, -1).nan_to_num_(0.0)
                out[starts[i]:starts[i + 1], j * g + m] = w @ v
    return out
