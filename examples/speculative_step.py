"""Speculative decoding steps around a paged 4-bit key/value cache.

Each step of every request, without a word from the host:

  draft     the Markov loop samples `drafts` tokens after the last one
  grow      room for the drafts and the last token in the page tables; a request that gets none sits the step out
  verify    the target model's layers over those rows: keys and values into the cache, attention over it
  accept    the longest run of drafts that the target agrees with, and its own next token
  trim      the cache is cut back to the rows that were kept

At the end some requests leave, the pool is compacted, and a request is forked into a free slot.

The target model is a toy with random weights (norm, projections, attention, projection, residual); what it shows is
the order of the calls and what passes between them.

    python examples/speculative_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dspark_markov_draft_anchor_gb300 import binding  # noqa: E402


class Target:
    """A toy target model: `layers` attention layers over embeddings of `vocab` tokens."""

    def __init__(self, vocab, hidden, layers, kv_heads, group, dim, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, device=device, generator=g) * n ** -0.5).bfloat16()
        self.kv_heads, self.group, self.dim = kv_heads, group, dim
        self.embed = torch.randn(vocab, hidden, device=device, generator=g).bfloat16()
        self.head = weight(hidden, vocab)
        wide = (kv_heads * group + 2 * kv_heads) * dim
        self.qkv = [weight(hidden, wide) for _ in range(layers)]
        self.out = [weight(kv_heads * group * dim, hidden) for _ in range(layers)]

    def norm(self, x):
        return torch.nn.functional.layer_norm(x, x.shape[-1:])

    def split(self, layer, x):
        """Queries, keys and values [rows, heads, dim]: views of one projection."""
        qh, kh = self.kv_heads * self.group, self.kv_heads
        y = (self.norm(x) @ self.qkv[layer]).unflatten(1, (qh + 2 * kh, self.dim))
        return y[:, :qh], y[:, qh:qh + kh], y[:, qh + kh:]


class Server:
    """Requests with their cache, and the calls of a step."""

    def __init__(self, target, requests, max_tokens, page_size, num_pages, drafts, device):
        self.target, self.requests, self.drafts, self.device = target, requests, drafts, device
        t, layers = target, len(target.qkv)
        pages = -(-max_tokens // page_size)
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device=device)
        self.table = torch.full((requests, pages), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.pool = binding.PagePool(self.refs, self.table, self.lens, page_size)
        size = binding.kv4_page_bytes(page_size, t.kv_heads, t.dim)
        self.data = torch.zeros(layers, num_pages, size, dtype=torch.uint8, device=device)
        self.caches = [binding.Kv4Cache(self.data[i], page_size, t.kv_heads, t.dim) for i in range(layers)]
        self.slots = torch.arange(requests, dtype=torch.int32, device=device)
        self.copy_src, self.copy_dst, self.granted = (torch.empty(requests, dtype=torch.int32, device=device)
                                                      for _ in range(3))
        self.workspace = torch.empty(0, dtype=torch.uint8, device=device)

    def grow(self, add):
        """Room for add[i] more tokens of request i where `granted` says so; shared last pages are copied in every
        layer."""
        binding.dspark_pages_grow(self.pool, self.slots, add, self.copy_src, self.copy_dst, self.granted)
        binding.dspark_pages_copy(self.data, self.copy_src, self.copy_dst)

    def forward(self, tokens, row_start, most):
        """The target's logits of the rows `tokens`, which are the newest ones of the requests that the last grow gave
        room to.  The others' rows belong to no slot: they are not stored and see nothing.  (Their cached tokens have
        not become more: as rows of their slots they would be stored over the last of them.)"""
        t = self.target
        slots = torch.where(self.granted > 0, self.slots, -1)
        batch = binding.Kv4Batch(row_start, self.lens, self.table, total_rows=tokens.numel(), max_rows=most, slots=slots)
        x = t.embed[tokens]
        size = binding.dspark_kv4_attention_workspace_bytes(self.caches[0], batch, t.kv_heads * t.group)
        if self.workspace.numel() < size:
            self.workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
        for i, cache in enumerate(self.caches):
            q, k, v = t.split(i, x)
            binding.dspark_kv4_append(cache, batch, k, v)
            y = torch.empty(q.shape, dtype=q.dtype, device=self.device)
            binding.dspark_kv4_attention(cache, batch, q, y, t.dim ** -0.5, self.workspace)
            x = x + y.flatten(1) @ t.out[i]
        return t.norm(x) @ t.head

    def prefill(self, prompts):
        """Prompts of any lengths into the cache; returns each one's next token."""
        sizes = [p.numel() for p in prompts]
        add = torch.tensor(sizes, dtype=torch.int32, device=self.device)
        row_start = torch.nn.functional.pad(torch.cumsum(add, 0), (1, 0)).int()
        self.grow(add)
        if not bool(self.granted.all()):  # the one word from the host, before the first step
            self.leave(self.slots)
            raise RuntimeError("the pool has no room for the prompts")
        logits = self.forward(torch.cat(prompts), row_start, max(sizes))
        return logits[(row_start[1:] - 1).long()].argmax(-1)

    def verify(self, last, draft):
        """One verification: accepted tokens [requests, drafts + 1] (-1 behind them) and how many (0 for a request
        without room, which is left as it was)."""
        b, p = draft.shape
        rows = torch.empty(b, p + 1, dtype=torch.int64, device=self.device)
        binding.dspark_build_verify_tokens(last, draft, rows, b, draft.stride(0), p)
        before = self.lens.clone()
        self.grow(torch.full((b,), p + 1, dtype=torch.int32, device=self.device))
        row_start = torch.arange(0, b * (p + 1) + 1, p + 1, dtype=torch.int32, device=self.device)
        logits = self.forward(rows.flatten(), row_start, p + 1)
        accepted = torch.empty(b, p + 1, dtype=torch.int64, device=self.device)
        count = torch.empty(b, dtype=torch.int32, device=self.device)
        wanted = torch.full((b,), p, dtype=torch.int32, device=self.device)
        binding.dspark_greedy_accept_noalloc(logits, draft, wanted, accepted, count, b, draft.stride(0), p,
                                             logits.shape[1])
        accepted.masked_fill_((self.granted == 0)[:, None], -1)
        count = count * self.granted
        # the last token and the accepted drafts stay; the token after them is next step's first row
        binding.dspark_pages_trim(self.pool, self.slots, before + count)
        return accepted, count

    def leave(self, slots):
        """Requests that have ended: their pages are freed."""
        binding.dspark_pages_trim(self.pool, slots, torch.zeros_like(slots))

    def compact(self):
        """The pages in use move to the pool's lowest ids; returns how many are in use."""
        to, src, dst = (torch.empty_like(self.refs) for _ in range(3))
        count = torch.empty(1, dtype=torch.int32, device=self.device)
        binding.dspark_pages_compact(self.pool, self.table, self.refs, to, src, dst, count)
        binding.dspark_pages_copy(self.data, src, dst, count=count)
        return (self.refs > 0).sum()

    def fork(self, src, dst):
        """Requests dst go on from where requests src are, on the same pages."""
        binding.dspark_pages_fork(self.pool, src, dst)

    def cached(self, layer, slot, tokens):
        """The last `tokens` cached keys and values of a request."""
        row_start = torch.tensor([0, tokens], dtype=torch.int32, device=self.device)
        slots = torch.tensor([slot], dtype=torch.int32, device=self.device)
        batch = binding.Kv4Batch(row_start, self.lens, self.table, total_rows=tokens, max_rows=tokens, slots=slots)
        t = self.target
        k = torch.empty(tokens, t.kv_heads, t.dim, dtype=torch.bfloat16, device=self.device)
        v = torch.empty_like(k)
        binding.dspark_kv4_read(self.caches[layer], batch, k, v)
        return k, v


def newest(accepted, count, before):
    """Each request's newest token: the last accepted one, or where there is none the one before."""
    last = accepted.gather(1, (count.long() - 1).clamp(min=0)[:, None])[:, 0]
    return torch.where(count > 0, last, before)


class Drafter:
    """The Markov draft loop over random tables and base logits."""

    def __init__(self, vocab, requests, drafts, device, seed=1):
        g = torch.Generator(device=device).manual_seed(seed)

        def bf16(*shape, scale):
            return (torch.randn(*shape, device=device, generator=g) * scale).bfloat16()
        self.w1, self.w2 = bf16(vocab, 256, scale=0.02), bf16(vocab, 256, scale=0.02)
        self.base = bf16(requests, drafts, vocab, scale=2.0)
        self.ctx = binding.MarkovContext(self.w1, self.w2, max_rows=requests, max_steps=drafts)
        self.index = torch.arange(requests, device=device)
        self.seeds = torch.arange(requests, device=device) + 77
        self.temperature = torch.zeros(requests, device=device)
        self.drafts, self.device = drafts, device

    def draft(self, last, lens):
        tokens = torch.empty(last.numel(), self.drafts, dtype=torch.int64, device=self.device)
        pos = lens.long()[:, None] + torch.arange(self.drafts, device=self.device)
        a = binding.loop_args(base=self.base, cache=None, input_ids=last.int(), anchor_idx=self.index, sample_pos=pos,
                              seeds=self.seeds, temperature=self.temperature, tokens=tokens)
        self.ctx.loop(a)
        return tokens


def main(requests=8, drafts=5, steps=6, vocab=4096, hidden=256, layers=2, kv_heads=2, group=4, dim=64, page_size=16,
         max_tokens=400, agree=0.7, seed=0, device="cuda"):
    """Runs `steps` verifications; returns the server and the tokens each request got.  The random tables seldom agree
    with the toy target, so a share `agree` of the drafts is replaced by what the target would say next."""
    g = torch.Generator(device=device).manual_seed(seed)
    target = Target(vocab, hidden, layers, kv_heads, group, dim, device, seed)
    server = Server(target, requests, max_tokens, page_size, requests * max_tokens // page_size, drafts, device)
    drafter = Drafter(vocab, requests, drafts, device)
    prompts = [torch.randint(0, vocab, (int(n),), device=device, generator=g)
               for n in torch.randint(1, 100, (requests,), generator=torch.Generator().manual_seed(seed))]
    last = server.prefill(prompts)
    got = [last[:, None]]
    for _ in range(steps):
        draft = drafter.draft(last, server.lens)
        for j in range(drafts):  # what the target says after the drafts so far, for a share of the places
            keep = server.lens.clone()
            accepted, count = server.verify(last, draft)
            say = newest(accepted, count, last)
            binding.dspark_pages_trim(server.pool, server.slots, keep)
            here = (count.long() - 1 == j) & (torch.rand(requests, device=device, generator=g) < agree)
            draft[:, j] = torch.where(here, say, draft[:, j])
        accepted, count = server.verify(last, draft)
        last = newest(accepted, count, last)
        got.append(accepted)
    return server, prompts, got


if __name__ == "__main__":
    server, prompts, got = main()
    kept = [(x >= 0).sum(1).tolist() for x in got[1:]]
    print("tokens of each request and step:", kept)
    print("cached tokens:", server.lens.tolist(), "pages held:", int((server.refs > 0).sum()))
    slots = server.slots[1::2].contiguous()
    server.leave(slots)
    print("pages held after every second request left:", int(server.compact()))
    server.fork(server.slots[:1], server.slots[1:2])
    print("cached tokens after forking request 0:", server.lens.tolist())
