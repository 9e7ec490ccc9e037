"""Operators of a long-context verification step: cases, inputs, plain forms and exact values.

Four operations between the target model's projections and the accept decision:

  append   rotate the step's queries and keys by their positions, store keys and values in their requests' 4-bit pages,
           and read back the values that the cache now stands for
  sparse   for each row and key/value head: bring the bounds of the step's pages up to date, score every page of the
           request by the largest product that its keys' bounds allow, keep `top` of them, attend over those
  count    admit requests: clear their slots of the token table, mark their prompts' tokens, count their outputs' ones
  adjust   a verification's logits: penalties for the tokens that a request (and the drafts before the row) already
           has, biases of single tokens, and a grammar's mask of the tokens that may come next

A page of the cache holds one record for each key/value head, `page * (dim + dim / 8)` bytes: key codes [page, dim / 2],
value codes [page, dim / 2], key scales [page, dim / 16], value scales [page, dim / 16]; byte j of a row of codes holds
element 2 j in its low four bits and 2 j + 1 in its high four (E2M1), a scale is E4M3 and serves 16 elements.  A page's
bounds hold for each head `2 * dim + 16` bytes: the smallest and the largest key code * scale of each dimension as int8
fractions (of 127) of the page's largest magnitude, [dim] and [dim], then that magnitude as FP32 and 12 bytes of zeros.
Rows of request i are row_start[i] .. row_start[i + 1] - 1; they are the last rows of its lens[i] cached ones.
"""
import random

import torch

own = False

LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of E2M1
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------

def _append(name, requests, rows, past, page, kv_heads, group, dim, rot, pairs="halves", dtype="bf16", scaled=False,
            given=False):
    return dict(name=name, op="append", requests=requests, rows_lo=rows[0], rows_hi=rows[1], past=past, page=page,
                kv_heads=kv_heads, group=group, dim=dim, rot=rot, pairs=pairs, dtype=dtype, scaled=scaled, given=given)


def _sparse(name, requests, rows, lens, page, kv_heads, group, dim, top, first=1, last=2, dtype="bf16", scaled=False):
    return dict(name=name, op="sparse", requests=requests, rows_lo=rows[0], rows_hi=rows[1], len_lo=lens[0],
                len_hi=lens[1], page=page, kv_heads=kv_heads, group=group, dim=dim, top=top, first=first, last=last,
                dtype=dtype, scaled=scaled)


def _count(name, requests, prompt, output, vocab, wide=True):
    return dict(name=name, op="count", requests=requests, prompt_lo=prompt[0], prompt_hi=prompt[1],
                output_lo=output[0], output_hi=output[1], vocab=vocab, wide=wide)


def _adjust(name, requests, drafts, vocab, held, dtype="bf16", out="f32", penalties=True, biases=0, masked=0.0):
    return dict(name=name, op="adjust", requests=requests, drafts=drafts, vocab=vocab, held=held, dtype=dtype, out=out,
                penalties=penalties, biases=biases, masked=masked)


def listed():
    return [
        # One request, one new token: latency counts.
        _append("append 1x1", 1, (1, 1), 2000, 64, 8, 8, 128, 128),
        # A verification of 16 requests with 5 drafts each.
        _append("append verify 16x6", 16, (6, 6), 4000, 64, 8, 8, 128, 128),
        # Prompts of mixed lengths entering the cache: neighbouring pairs, half of each head rotated, positions of the
        # caller's own (a prompt after a shared prefix), a calibrated scale for each head.
        _append("append prompts", 12, (1, 4001), 1000, 32, 8, 8, 128, 64, "neighbours", "bf16", True, True),
        # One request with a long context, one token.
        _sparse("sparse 1x1 128k", 1, (1, 1), (131072, 131072), 64, 8, 8, 128, 64),
        # Decoding a batch of long requests, one token each.
        _sparse("sparse 32x1 64k", 32, (1, 1), (16384, 65536), 64, 8, 8, 128, 64),
        # The verification of 5 drafts (6 rows) over long contexts.
        _sparse("sparse verify 16x6 32k", 16, (6, 6), (8192, 32768), 64, 8, 8, 128, 32),
        # A mixed step of odd sizes: idle requests, some shorter than the pages that are kept, an odd group, small
        # heads and pages, head scales.
        _sparse("sparse mixed odd", 23, (0, 17), (0, 9001), 16, 5, 5, 64, 33, 2, 3, "f16", True),
        # A few short requests come back after a preemption.
        _count("count 3 short", 3, (1, 900), (0, 300), 32768),
        # A batch of long prompts is admitted.
        _count("count 64 long", 64, (1001, 32001), (0, 2000), 129280, False),
        # Decoding one request: penalties for what it holds, a few biases, no grammar.
        _adjust("adjust 1x1", 1, 0, 129280, 2000, "bf16", "f32", True, 20, 0.0),
        # The verification of 5 drafts for a batch, a third of the requests under a grammar.
        _adjust("adjust verify 64x6", 64, 5, 163840, 3000, "bf16", "f32", True, 50, 0.33),
        # Odd sizes, FP32 in and out, every request under a grammar (one of whose masks leaves nothing).
        _adjust("adjust odd 23x4", 23, 3, 50021, 700, "f32", "f32", True, 7, 1.0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, odd above 16."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return min(hi, v | 1) if v > 16 else v


def draw(rng):
    op = rng.choice(("append", "append", "sparse", "sparse", "sparse", "count", "adjust", "adjust"))
    page = rng.choice((16, 32, 64, 128))
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    group = rng.choice((1, 2, 4, 5, 7, 8))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    scaled = rng.random() < 0.5
    if op == "append":
        requests = _log(rng, 1, 200)
        rows = _log(rng, 1, max(2, 20000 // requests))
        c = _append("", requests, (rng.choice((1, rows)) if rows < 40 else 1, rows), _log(rng, 1, 4001), page,
                    kv_heads, group, dim, rng.choice([n for n in (32, 64, 96, 128) if n <= dim]),
                    rng.choice(("halves", "halves", "neighbours")), dtype, scaled, rng.random() < 0.3)
    elif op == "sparse":
        kind = rng.choice(("one", "verify", "verify", "chunk"))
        requests = _log(rng, 1, {"one": 101, "verify": 41, "chunk": 5}[kind])
        lens = _log(rng, 17, min(131071, 1000000 // requests))
        rows = {"one": (1, 1), "verify": (rng.choice((0, 1, 2)), rng.choice((2, 4, 6, 8))),
                "chunk": (1, _log(rng, 9, 65))}[kind]
        first, last = rng.choice((0, 1, 2)), rng.choice((1, 2, 4))
        top = max(first + last, _log(rng, 3, 129))
        if page == 128:
            top = min(top, 64)
        c = _sparse("", requests, rows, (rng.choice((0, lens // 2, lens)), lens), page, kv_heads, group, dim, top,
                    first, last, dtype, scaled)
    elif op == "count":
        requests = _log(rng, 1, 64)
        c = _count("", requests, (rng.choice((0, 1, 50)), _log(rng, 51, 32001)), (0, _log(rng, 1, 2001)),
                   _log(rng, 1000, 129280), rng.random() < 0.5)
    else:
        requests, drafts = _log(rng, 1, 64), rng.choice((0, 0, 1, 3, 5, 7))
        vocab = _log(rng, 1000, 163840)
        if rng.random() < 0.5:
            vocab = max(8, vocab // 8 * 8)
        while requests * (drafts + 1) * vocab > 384 * 163840:
            requests = max(1, requests // 2)
        kind, out = rng.choice((("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")))
        c = _adjust("", requests, drafts, vocab, _log(rng, 1, max(1, min(4000, vocab // 2))), kind, out,
                    rng.random() < 0.8, rng.choice((0, 1, 10, 60)), rng.choice((0.0, 0.5, 1.0)))
    del c["name"]
    return c


def _record(c):
    """Bytes of one head's record of a page."""
    return c["page"] * (c["dim"] + c["dim"] // 8)


def _pages(n, page):
    return -(-n // page)


def _shape(c):
    """Rows and lengths of a case's requests (prompt and output lengths, for count): the same whatever the seed, so
    that outputs of two seeds have one shape."""
    rng = random.Random(",".join("%s=%s" % (k, c[k]) for k in sorted(c) if k != "name"))
    n = c["requests"]
    if c["op"] == "count":
        return ([rng.randint(c["prompt_lo"], c["prompt_hi"]) for _ in range(n)],
                [rng.randint(c["output_lo"], c["output_hi"]) for _ in range(n)])
    if c["op"] == "append":
        rows = [rng.randint(c["rows_lo"], c["rows_hi"]) for _ in range(n)]
        return rows, [rng.randint(0, c["past"]) + r for r in rows]
    lens = [rng.randint(c["len_lo"], c["len_hi"]) for _ in range(n)]
    rows = [rng.randint(c["rows_lo"], c["rows_hi"]) for _ in range(n)]
    if c["len_lo"]:  # else some requests have more rows than cached tokens: rows that see nothing
        rows = [min(r, t) for r, t in zip(rows, lens)]
    rows[-1] = max(rows[-1], 1)
    return rows, lens


def _masked(c):
    """How many requests of an adjust case are under a grammar."""
    return int(round(c["masked"] * c["requests"]))


def work(case):
    c = case
    if c["op"] == "adjust":
        b, r, v = c["requests"], c["drafts"] + 1, c["vocab"]
        size = {"bf16": 2, "f32": 4}
        held = b * (c["held"] * 4 * c["penalties"] + c["biases"] * 8)
        return {"bytes": b * r * v * (size[c["dtype"]] + size[c["out"]]) + _masked(c) * r * v / 8 +
                b * v / 4 * c["penalties"] + held, "flops": b * r * (c["held"] * 4 + c["biases"])}
    rows, lens = _shape(c)
    if c["op"] == "count":
        size = 8 if c["wide"] else 4
        return {"bytes": c["requests"] * c["vocab"] * (4 + 1 / 4) + (sum(rows) + sum(lens)) * size, "flops": 0}
    h, g, d, page = c["kv_heads"], c["group"], c["dim"], c["page"]
    if c["op"] == "append":
        # keys and values in, codes and scales out, the same back for the read; queries in and out; the table's rows
        n = sum(rows)
        return {"bytes": n * (h * d * 2 * (2 + 9 / 16) * 2 + h * g * d * 4 + c["rot"] * 4),
                "flops": n * (h * d * 4 + 3 * h * (g + 1) * c["rot"])}
    size = flops = 0
    for n, t in zip(rows, lens):
        if n == 0 or t == 0:
            continue
        touched = _pages(t, page) - max(0, t - n) // page
        total = _pages(t, page)
        # each page's bounds; the step's pages' keys and new bounds; queries in, results out, the lists
        size += total * h * (2 * d + 16) + touched * h * (page * d * 9 / 16 + 2 * d + 16)
        size += n * (h * g * d * 4 + h * c["top"] * 4 + 4)
        kept = min(c["top"], total)
        # of the pages that are kept, at least those that one row keeps have to be read
        size += kept * h * _record(c)
        flops += n * h * (total * 4 * d + min(kept * page, t) * g * d * 4)
    return {"bytes": size, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------------
# The plain form of the cache: quantising, storing and reading, 32-bit arithmetic on torch operations
# ---------------------------------------------------------------------------------------------------------------------

def _quantise(x, g):
    """x [..., heads, dim] -> codes (uint8, one a value), scales (uint8 E4M3, one for 16); g: [heads] or None."""
    y = x.float()
    if g is not None:
        y = y / g[:, None]
    y = y.reshape(*x.shape[:-1], -1, 16)
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
    """The four sections of pages' bytes [pages, heads * record] as views: key codes, value codes, key scales, value
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


def _bounds(keys, there):
    """Bounds of pages: keys [pages, heads, page, dim] without the heads' scales, there [pages, page] -> the int8
    fractions [pages, heads, 2 * dim] and the magnitudes [pages, heads]."""
    gone = ~there[:, None, :, None]
    lo = keys.masked_fill(gone, torch.inf).amin(2)
    hi = keys.masked_fill(gone, -torch.inf).amax(2)
    both = torch.cat((lo, hi), -1)
    top = both.abs().amax(-1)
    part = torch.round(both * 127.0 / torch.where(top > 0, top, torch.ones_like(top))[..., None])
    return part.to(torch.int8), top


def _put_bounds(bounds, c, ids, part, top):
    """Bounds into the pages' bytes [num_pages, heads * (2 * dim + 16)]."""
    rec = torch.zeros(*top.shape, 2 * c["dim"] + 16, dtype=torch.uint8, device=bounds.device)
    rec[..., :2 * c["dim"]] = part.view(torch.uint8)
    rec[..., 2 * c["dim"]:2 * c["dim"] + 4] = top.contiguous().view(torch.uint8).unflatten(-1, (-1, 4))
    bounds[ids] = rec.flatten(1)


def _keys(data, c, ids):
    """The keys of pages `ids` without the heads' scales, FP32 [pages, heads, page, dim]."""
    kc, _, ks, _ = _sections(data[ids], c)
    code = torch.stack((kc & 15, kc >> 4), -1).flatten(-2)
    return _values(code, ks.contiguous(), None)


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
    if c["op"] == "count":
        return _prepare_count(c, gen)
    if c["op"] == "adjust":
        return _prepare_adjust(c, gen)
    cpu = torch.Generator().manual_seed(seed)
    dtype, h, d, b = TYPES[c["dtype"]], c["kv_heads"], c["dim"], c["requests"]
    rows, lens = _shape(c)
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
             gk=scales[0], gv=scales[1], total=total, most=max(rows), rows=rows, tokens=lens,
             data=torch.randint(0, 256, (num_pages, h * _record(c)), dtype=torch.uint8, device="cuda", generator=gen))
    s["q"] = _rows(total, h * c["group"], d, dtype, gen, 0.4)
    if c["op"] == "append":
        s["k"] = _rows(total, h, d, dtype, gen, 0.7)
        s["v"] = _rows(total, h, d, dtype, gen, 0.3)
        s["k_seen"], s["v_seen"], s["q_out"] = (torch.empty_like(s[n]) for n in ("k", "v", "q"))
        far = max(lens) + 700
        angle = torch.arange(far, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["given"] = None
        if c["given"]:  # the cached rows' positions begin at 700: a prefix that the cache does not hold
            s["given"] = (_owner(s)[1] + 700).int()
    else:
        for at in range(0, num_pages, 1024):  # a cache that earlier steps filled; a page's keys lie around a centre
            part = s["data"][at:at + 1024]
            n = part.shape[0] * c["page"]
            page_of = torch.arange(n, device="cuda") // c["page"]
            row_of = torch.arange(n, device="cuda") % c["page"]
            k = _rows(part.shape[0], h, d, torch.float32, gen, 0.4)[page_of] * 0.7 + _rows(n, h, d, torch.float32, gen, 0.4)
            _store(part, c, page_of, row_of, k, _rows(n, h, d, dtype, gen, 0.3), s["gk"], s["gv"])
        s["bounds"] = torch.zeros(num_pages, h * (2 * d + 16), dtype=torch.uint8, device="cuda")
        whole = torch.ones(1, c["page"], dtype=torch.bool, device="cuda")
        for at in range(0, num_pages, 1024):
            some = torch.arange(at, min(at + 1024, num_pages), device="cuda")
            _put_bounds(s["bounds"], c, some, *_bounds(_keys(s["data"], c, some), whole))
        rec = s["bounds"].unflatten(1, (h, -1))  # seen as the numbers that they hold
        s["parts"], s["sizes"] = rec[..., :2 * d].view(torch.int8), rec.view(torch.float32)[..., d // 2]
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = d ** -0.5
        s["pages"] = torch.empty(total, h, c["top"], dtype=torch.int32, device="cuda")
        s["kept"] = torch.empty(total, dtype=torch.int32, device="cuda")
    if own:
        from dspark_markov_draft_anchor_gb300 import binding
        s["cache"] = binding.Kv4Cache(s["data"], c["page"], h, d, k_scale=s["gk"], v_scale=s["gv"])
        s["batch"] = binding.Kv4Batch(s["row_start"], s["lens"], s["table"], total_rows=total, max_rows=s["most"])
        if c["op"] == "append":
            s["rotation"] = binding.Kv4Rotation(s["cos"], s["sin"], interleaved=c["pairs"] == "neighbours",
                                                positions=s["given"])
        else:
            s["selection"] = binding.Kv4Selection(s["pages"], s["kept"])
            size = max(binding.dspark_kv4_select_workspace_bytes(s["cache"], s["batch"], s["selection"]),
                       binding.dspark_kv4_attention_selected_workspace_bytes(s["cache"], s["selection"],
                                                                             h * c["group"]))
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _words(vocab):
    return -(-vocab // 32)


def _tokens(n, width, vocab, gen):
    """Token ids as texts have them: a few often, most seldom."""
    u = torch.rand(n, width, device="cuda", generator=gen)
    return (vocab ** u.double() - 1).long().clamp(max=vocab - 1) * 7919 % vocab


def _prepare_count(c, gen):
    b, v = c["requests"], c["vocab"]
    prompts, outputs = _shape(c)
    kind = torch.int64 if c["wide"] else torch.int32
    s = dict(c=c, prompt=_tokens(b, max(1, max(prompts)), v, gen).to(kind),
             output=_tokens(b, max(1, max(outputs)), v, gen).to(kind), prompts=_ints(prompts), outputs=_ints(outputs),
             slots=torch.randperm(b, device="cuda", generator=gen).int(),
             counts=torch.randint(0, 5, (b, v), dtype=torch.int32, device="cuda", generator=gen),  # a request before
             marks=torch.randint(-2 ** 31, 2 ** 31, (b, 2, _words(v)), device="cuda", generator=gen).int())
    if own:
        from dspark_markov_draft_anchor_gb300 import binding
        s["tokens"] = binding.TokenTable(s["counts"], s["marks"])
    return s


def _bits(flags):
    """Truth values [..., n] as int32 words, bit i % 32 of word i / 32."""
    n = flags.shape[-1]
    f = torch.nn.functional.pad(flags, (0, -n % 32)).unflatten(-1, (-1, 32)).long()
    w = (f << torch.arange(32, device=flags.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def _prepare_adjust(c, gen):
    b, r, v = c["requests"], c["drafts"] + 1, c["vocab"]
    s = dict(c=c, logits=(torch.randn(b * r, v, device="cuda", generator=gen) * 3).to(TYPES[c["dtype"]]),
             slots=torch.randperm(b, device="cuda", generator=gen).int(), draft=None, repetition=None, frequency=None,
             presence=None, bias=None, mask=None, mask_rows=None)
    s["out"] = torch.empty(b * r, v, dtype=TYPES[c["out"]], device="cuda")
    counts = torch.zeros(b, v, dtype=torch.int32, device="cuda")
    held = _tokens(b, c["held"], v, gen)
    split = c["held"] // 2  # prompt first, then outputs
    counts.scatter_add_(1, held[:, split:], torch.ones_like(held[:, split:], dtype=torch.int32))
    prompt = torch.zeros(b, v, dtype=torch.bool, device="cuda").scatter_(1, held[:, :split], True)
    s["counts"], s["marks"] = counts, _bits(torch.stack((prompt, counts > 0), 1))
    if c["drafts"]:
        s["draft"] = _tokens(b, c["drafts"], v, gen)
    if c["penalties"]:
        s["repetition"] = torch.empty(b, device="cuda").uniform_(1.0, 1.4, generator=gen)
        s["frequency"] = torch.empty(b, device="cuda").uniform_(-0.1, 0.5, generator=gen)
        s["presence"] = torch.empty(b, device="cuda").uniform_(0.0, 0.6, generator=gen)
    if c["biases"]:
        n = min(c["biases"], v)
        ids = torch.stack([torch.randperm(v, device="cuda", generator=gen)[:n] for _ in range(b)]).int().flatten()
        s["bias"] = (_ints(range(0, b * n + 1, n)), ids, torch.randn(b * n, device="cuda", generator=gen) * 4)
    m = _masked(c)
    if m:  # a few states of a grammar: some allow most tokens, some a few, one none
        share = torch.empty(m * r, 1, device="cuda").uniform_(0.0, 1.0, generator=gen)
        share = torch.where(share < 0.5, torch.full_like(share, 50.0 / v), 0.5 + share / 2)
        share[-1] = 0.0
        allowed = torch.rand(m * r, v, device="cuda", generator=gen) < share
        s["mask"] = _bits(allowed)
        s["mask_rows"] = _ints([i * r + j if i < m else -1 for i in range(b) for j in range(r)])
    if own:
        from dspark_markov_draft_anchor_gb300 import binding
        s["tokens"] = binding.TokenTable(s["counts"], s["marks"])
    return s


# ---------------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        return {"append": _own_append, "sparse": _own_sparse, "count": _own_count, "adjust": _own_adjust}[op](s)
    return {"append": _plain_append, "sparse": _plain_sparse, "count": _plain_count, "adjust": _plain_adjust}[op](s)


def _own_append(s):
    from dspark_markov_draft_anchor_gb300 import binding
    binding.dspark_kv4_append_rotated(s["cache"], s["batch"], s["rotation"], s["k"], s["v"], s["q"], s["q_out"])
    binding.dspark_kv4_read(s["cache"], s["batch"], s["k_seen"], s["v_seen"])
    return s["q_out"], s["k_seen"], s["v_seen"]


def _own_sparse(s):
    from dspark_markov_draft_anchor_gb300 import binding
    c = s["c"]
    binding.dspark_kv4_bound_pages(s["cache"], s["batch"], s["bounds"])
    binding.dspark_kv4_select(s["cache"], s["batch"], s["bounds"], s["q"], s["selection"], s["workspace"],
                              first=c["first"], last=c["last"])
    binding.dspark_kv4_attention_selected(s["cache"], s["selection"], s["q"], s["out"], s["scale"], s["workspace"])
    return s["pages"], s["kept"], s["out"], s["parts"], s["sizes"]


def _own_count(s):
    from dspark_markov_draft_anchor_gb300 import binding
    binding.dspark_tokens_count(s["tokens"], s["prompt"], s["prompts"], slots=s["slots"], prompt=True, reset=True)
    binding.dspark_tokens_count(s["tokens"], s["output"], s["outputs"], slots=s["slots"])
    return s["counts"], s["marks"]


def _own_adjust(s):
    from dspark_markov_draft_anchor_gb300 import binding
    binding.dspark_logits_adjust(s["tokens"], s["logits"], s["out"], drafts=s["c"]["drafts"], slots=s["slots"],
                                 draft=s["draft"], repetition=s["repetition"], frequency=s["frequency"],
                                 presence=s["presence"], bias=s["bias"], mask=s["mask"], mask_rows=s["mask_rows"])
    return s["out"]


def _owner(s):
    """For each row: its request, and its position in the request's cache."""
    start, total = s["row_start"].long(), s["total"]
    row = torch.arange(total, device="cuda")
    owner = torch.searchsorted(start[1:], row, right=True)
    return owner, row - start[owner + 1] + s["lens"].long()[owner]


def _rotate(x, cos, sin, c):
    """x [rows, heads, dim], cos and sin [rows, rot / 2] -> FP32."""
    x, r = x.float(), c["rot"]
    cos, sin = cos[:, None], sin[:, None]
    out = x.clone()
    if c["pairs"] == "halves":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        out[..., :r // 2], out[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return out


def _plain_append(s):
    c = s["c"]
    owner, pos = _owner(s)
    at = pos if s["given"] is None else s["given"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    page_of = s["table"].long()[owner, pos // c["page"]]
    (kc, ks), (vc, vs) = _store(s["data"], c, page_of, pos % c["page"], _rotate(s["k"], cos, sin, c), s["v"], s["gk"],
                                s["gv"])
    dtype = TYPES[c["dtype"]]
    return (_rotate(s["q"], cos, sin, c).to(dtype), _values(kc, ks, s["gk"]).to(dtype),
            _values(vc, vs, s["gv"]).to(dtype))


def _query_parts(q, gk):
    """The queries of a head's group as one int8 vector for each row and head: what meets a page's smallest keys, then
    what meets its largest.  q [rows, heads, group, dim]."""
    x = q.float().clamp(-2.0 ** 100, 2.0 ** 100)
    if gk is not None:
        x = x * torch.sign(gk)[:, None, None]
    parts = []
    for y in (x.clamp(max=0.0), x.clamp(min=0.0)):
        t = y[:, :, 0]
        for m in range(1, y.shape[2]):
            t = t + y[:, :, m]
        parts.append(t)
    both = torch.cat(parts, -1)
    top = both.abs().amax(-1, keepdim=True)
    return torch.round(both * 127.0 / torch.where(top > 0, top, torch.ones_like(top)))


def _plain_sparse(s):
    c = s["c"]
    h, g, d, page, top = c["kv_heads"], c["group"], c["dim"], c["page"], c["top"]
    s["pages"].fill_(-1)
    s["kept"].zero_()
    s["out"].zero_()
    at = 0
    for i, (n, t) in enumerate(zip(s["rows"], s["tokens"])):
        start, at = at, at + n
        if n == 0 or t == 0:
            continue
        ids = s["table"][i, :_pages(t, page)].long()
        # bounds of the pages that the step's rows are in
        low = max(0, t - n) // page
        there = torch.arange(low * page, ids.numel() * page, device="cuda").unflatten(0, (-1, page)) < t
        _put_bounds(s["bounds"], c, ids[low:], *_bounds(_keys(s["data"], c, ids[low:]), there))
        # scores
        skip = max(0, n - t)  # rows that see nothing
        q = s["q"][start + skip:at].unflatten(1, (h, g))
        rec = s["bounds"][ids].unflatten(1, (h, -1))
        part = rec[..., :2 * d].contiguous().view(torch.int8).float()
        size = rec[..., 2 * d:2 * d + 4].contiguous().view(torch.float32)[..., 0]
        score = torch.einsum("nhd,phd->nhp", _query_parts(q, s["gk"]), part) * size.T
        pos = torch.arange(t - n + skip, t, device="cuda")
        here = (pos // page + 1)[:, None, None]  # pages of each row
        p = torch.arange(ids.numel(), device="cuda")
        score = score.masked_fill((p < c["first"]) | (p >= here - c["last"]), torch.inf)
        score = score.masked_fill(p >= here, -torch.inf)
        # the `top` largest, ties to the lowest page; in ascending order
        order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
        count = here.clamp(max=top)
        nth = torch.arange(order.shape[-1], device="cuda")
        order = torch.where(nth < count, order, torch.full_like(order, 2 ** 40)).sort(-1).values
        some = nth < count
        picked = torch.where(some, ids[order.clamp(max=ids.numel() - 1)], torch.full_like(order, -1))
        s["pages"][start + skip:at, :, :order.shape[-1]] = picked.int()
        kept = (count[:, 0, 0] - 1) * page + pos % page + 1
        s["kept"][start + skip:at] = kept.int()
        # attention
        head = torch.arange(h, device="cuda")[:, None]
        data = s["data"].unflatten(1, (h, -1))
        rec = data[picked.clamp(min=0), head]  # [rows, heads, top, record]
        one = dict(c, kv_heads=1)
        kc, vc, ks, vs = _sections(rec.flatten(0, 2), one)
        both = []
        for codes, scales, w in ((kc, ks, s["gk"]), (vc, vs, s["gv"])):
            code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
            x = _values(code, scales.contiguous(), None).reshape(*picked.shape[:2], -1, d)
            both.append(x if w is None else x * w[:, None, None])
        k, v = both
        sc = (q.float() @ k.transpose(2, 3)) * s["scale"]
        seen = torch.arange(k.shape[2], device="cuda") < kept[:, None]
        sc = sc.masked_fill(~seen[:, None, None], -torch.inf)
        w = torch.exp(sc - sc.amax(-1, keepdim=True))
        y = (w @ v) / w.sum(-1, keepdim=True)
        s["out"][start + skip:at] = y.flatten(1, 2).to(s["out"].dtype)
    return s["pages"], s["kept"], s["out"], s["parts"], s["sizes"]


def _plain_count(s):
    c = s["c"]
    v = c["vocab"]
    slots = s["slots"].long()
    seen = []
    for tokens, lens in ((s["prompt"], s["prompts"]), (s["output"], s["outputs"])):
        here = torch.arange(tokens.shape[1], device="cuda") < lens[:, None]
        n = torch.zeros(c["requests"], v, dtype=torch.int32, device="cuda")
        seen.append(n.scatter_add_(1, tokens.long(), here.int()))
    s["counts"][slots] = seen[1]
    s["marks"][slots] = _bits(torch.stack((seen[0] > 0, seen[1] > 0), 1))
    return s["counts"], s["marks"]


def _flags(words, n):
    """The truth values of int32 words."""
    return ((words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1).flatten(-2)[..., :n] != 0


def _plain_adjust(s):
    c = s["c"]
    b, r, v = c["requests"], c["drafts"] + 1, c["vocab"]
    slots = s["slots"].long()
    x = s["logits"].float().unflatten(0, (b, r))
    if c["penalties"]:
        n = s["counts"][slots][:, None].repeat(1, r, 1)
        for j in range(1, r):  # the drafts before row j
            here = torch.ones(b, r - j, 1, dtype=torch.int32, device="cuda")
            n[:, j:].scatter_add_(2, s["draft"][:, None, j - 1:j].expand(-1, r - j, -1), here)
        prompt = _flags(s["marks"][slots, 0], v)[:, None]
        rep, freq, pres = (s[k][slots][:, None, None] for k in ("repetition", "frequency", "presence"))
        x = torch.where(prompt | (n > 0), torch.where(x > 0, x / rep, x * rep), x)
        x = torch.where(n > 0, x - freq * n - pres, x)
    if s["bias"] is not None:
        start, ids, values = s["bias"]
        per = ids.numel() // b
        dense = torch.zeros(b, v, device="cuda").scatter_(1, ids.long().reshape(b, per), values.reshape(b, per))
        x = x + dense[slots][:, None]
    x = x.flatten(0, 1)
    if s["mask"] is not None:
        at = s["mask_rows"].long()
        x = torch.where((at >= 0)[:, None] & ~_flags(s["mask"], v)[at.clamp(min=0)], torch.full_like(x, -torch.inf), x)
    s["out"].copy_(x)
    return s["out"]


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
    if c["op"] == "count":
        return None
    s = prepare(c, seed)
    return {"append": _exact_append, "sparse": _exact_sparse, "adjust": _exact_adjust}[c["op"]](s)


def _exact_append(s):
    c = s["c"]
    pos = s["given"]
    if pos is None:
        pos = torch.cat([torch.arange(t - n, t) for n, t in zip(s["rows"], s["tokens"])]).cuda()
    pos = pos.long()
    r = c["rot"]
    w = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
    turned = []
    for x in (s["q"].double(), s["k"].double()):
        if c["pairs"] == "halves":
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * w
            y = torch.cat((z.real, z.imag, x[..., r:]), -1)
        else:
            z = torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous()) * w
            y = torch.cat((torch.view_as_real(z).flatten(-2), x[..., r:]), -1)
        turned.append(y)
    return turned[0], _quantised64(turned[1], s["gk"]), _quantised64(s["v"], s["gv"])


def _exact_sparse(s):
    c = s["c"]
    h, g, d, page, top = c["kv_heads"], c["group"], c["dim"], c["page"], c["top"]
    if sum(s["rows"]) * h * top > 200000:
        return None
    half, eighth = page * d // 2, page * d // 16
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    parts, sizes = s["parts"].clone(), s["sizes"].double()

    def cached(pages, j, at, sc):
        """[pages * page, dim] of head j, without its scale."""
        rec = s["data"][pages, j * _record(c):(j + 1) * _record(c)].int()
        byte = rec[:, at:at + half].reshape(-1, d // 2)
        x = torch.empty(byte.shape[0], d, dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = _nibble64(byte & 15), _nibble64(byte >> 4)
        return x * _e4m3_64(rec[:, sc:sc + eighth].reshape(-1, d // 16)).repeat_interleave(16, 1)

    kept = [0] * s["total"]  # tokens of the pages that a row keeps
    at = 0
    for i, (n, t) in enumerate(zip(s["rows"], s["tokens"])):
        start, at = at, at + n
        if n == 0 or t == 0:
            continue
        for m in range(max(0, n - t), n):
            pos = t - n + m
            kept[start + m] = min(pos + 1, (top - 1) * page + pos % page + 1)
        ids = s["table"][i, :_pages(t, page)].long()
        for j in range(h):
            gk = 1.0 if s["gk"] is None else s["gk"][j].double()
            gv = 1.0 if s["gv"] is None else s["gv"][j].double()
            lo, hi = [], []
            for first in range(0, ids.numel(), 512):  # each page's bounds, from its keys
                k = cached(ids[first:first + 512], j, 0, 2 * half).unflatten(0, (-1, page))
                live = (torch.arange(k.shape[0] * page, device="cuda") + first * page).unflatten(0, (-1, page)) < t
                lo.append(torch.where(live[..., None], k, torch.inf).amin(1))
                hi.append(torch.where(live[..., None], k, -torch.inf).amax(1))
            lo, hi = torch.cat(lo), torch.cat(hi)
            size = torch.maximum(lo.abs().amax(1), hi.abs().amax(1))
            unit = size.clamp(min=1e-300)[:, None]
            lo, hi = torch.round(lo * 127 / unit), torch.round(hi * 127 / unit)
            low = max(0, t - n) // page  # the step's pages: their bounds are new
            parts[ids[low:], j], sizes[ids[low:], j] = torch.cat((lo, hi), 1)[low:].to(torch.int8), size[low:]
            for m in range(max(0, n - t), n):
                pos = t - n + m
                here = pos // page + 1
                q = s["q"][start + m, j * g:(j + 1) * g].double()
                a, b = q.clamp(max=0.0).sum(0), q.clamp(min=0.0).sum(0)
                most = max(float(a.abs().max()), float(b.max()), 1e-300)
                a, b = torch.round(a * 127 / most), torch.round(b * 127 / most)
                score = (size * (lo @ a + hi @ b))[:here].clone()
                score[:c["first"]] = torch.inf
                score[max(0, here - c["last"]):] = torch.inf
                keep = torch.sort(score, descending=True, stable=True).indices[:top].sort().values
                k = cached(ids[keep], j, 0, 2 * half)
                v = cached(ids[keep], j, half, 2 * half + eighth)
                live = (keep[:, None] * page + torch.arange(page, device="cuda")).flatten() <= pos
                w = (q @ k.T) * gk * s["scale"]
                w = torch.softmax(torch.where(live, w, -torch.inf), -1)
                out[start + m, j * g:(j + 1) * g] = (w @ v) * gv
    return None, s["kept"].new_tensor(kept), out, parts, sizes


def _exact_adjust(s):
    c = s["c"]
    r = c["drafts"] + 1
    x = s["logits"].double()
    for i, slot in enumerate(s["slots"].tolist()):
        for j in range(r):
            y = x[i * r + j]
            if c["penalties"]:
                n = s["counts"][slot].double()
                if j:
                    n = n + torch.bincount(s["draft"][i, :j], minlength=c["vocab"])
                bit = torch.arange(c["vocab"], device="cuda")
                held = (s["marks"][slot, 0].long()[bit // 32] >> (bit % 32)) % 2 == 1
                rep = s["repetition"][slot].double()
                y = torch.where(held | (n > 0), torch.where(y > 0, y / rep, y * rep), y)
                y = y - s["frequency"][slot].double() * n - s["presence"][slot].double() * (n > 0)
            if s["bias"] is not None:
                first, last = s["bias"][0][slot:slot + 2].tolist()
                y = y.index_add(0, s["bias"][1][first:last].long(), s["bias"][2][first:last].double())
            if s["mask"] is not None and int(s["mask_rows"][i * r + j]) >= 0:
                word = s["mask"][s["mask_rows"][i * r + j].long()].long()
                bit = torch.arange(c["vocab"], device="cuda")
                y = torch.where((word[bit // 32] >> (bit % 32)) % 2 == 1, y, -torch.inf)
            x[i * r + j] = y
    return x
