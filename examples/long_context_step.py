"""Speculative decoding steps over long contexts: the steps of speculative_step.py with

  rotation   queries and keys are turned by their positions, keys on their way into the 4-bit cache
  selection  a verification's rows attend to a few pages of the cache each, chosen by the bounds of the pages' keys
             (prompts attend to everything)
  logits     penalties for what a request has said (and for the drafts before a row), biases, and masks of the tokens
             that may come, between the target's logits and the accept

    python examples/long_context_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import speculative_step  # noqa: E402
from speculative_step import Drafter, Target, binding, newest  # noqa: E402


class Server(speculative_step.Server):
    """top, first, last: pages that a row attends to, and how many of them are the request's first and last ones.
    presence, repetition: of every request.  allowed: truth values [vocab], the tokens that may be said, or None."""

    def __init__(self, target, requests, max_tokens, page_size, num_pages, drafts, device, *, top=8, first=1, last=2,
                 presence=0.0, repetition=1.0, allowed=None):
        super().__init__(target, requests, max_tokens, page_size, num_pages, drafts, device)
        t = target
        vocab, layers = t.embed.shape[0], len(t.qkv)
        self.top, self.first, self.last = top, first, last
        angle = torch.arange(max_tokens, device=device)[:, None] * 10000.0 ** (
            -torch.arange(0, t.dim, 2, dtype=torch.float64, device=device) / t.dim)
        self.rotation = binding.Kv4Rotation(angle.cos().float(), angle.sin().float())
        self.bounds = torch.zeros(layers, num_pages, binding.kv4_bounds_bytes(t.kv_heads, t.dim), dtype=torch.uint8,
                                  device=device)
        words = -(-vocab // 32)
        self.said = binding.TokenTable(torch.zeros(requests, vocab, dtype=torch.int32, device=device),
                                       torch.zeros(requests, 2, words, dtype=torch.int32, device=device))
        self.presence = torch.full((requests,), presence, device=device)
        self.repetition = torch.full((requests,), repetition, device=device)
        self.mask = None
        if allowed is not None:
            bits = torch.nn.functional.pad(allowed, (0, 32 * words - vocab)).unflatten(0, (words, 32)).long()
            bits = (bits << torch.arange(32, device=device)).sum(-1)
            self.mask = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).int()[None]

    def room(self, size):
        if self.workspace.numel() < size:
            self.workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
        return self.workspace

    def forward(self, tokens, row_start, most):
        t, rows = self.target, tokens.numel()
        heads = t.kv_heads * t.group
        slots = torch.where(self.granted > 0, self.slots, -1)
        batch = binding.Kv4Batch(row_start, self.lens, self.table, total_rows=rows, max_rows=most, slots=slots)
        few = most <= self.drafts + 1  # a verification; prompts attend to all of their tokens
        if few:
            selection = binding.Kv4Selection(
                torch.empty(rows, t.kv_heads, self.top, dtype=torch.int32, device=self.device),
                torch.empty(rows, dtype=torch.int32, device=self.device))
        x = t.embed[tokens]
        for i, cache in enumerate(self.caches):
            q, k, v = t.split(i, x)
            turned, y = torch.empty(q.shape, dtype=q.dtype, device=self.device), torch.empty(q.shape, dtype=q.dtype, device=self.device)
            binding.dspark_kv4_append_rotated(cache, batch, self.rotation, k, v, q, turned)
            binding.dspark_kv4_bound_pages(cache, batch, self.bounds[i])
            if few:
                work = self.room(max(binding.dspark_kv4_select_workspace_bytes(cache, batch, selection),
                                     binding.dspark_kv4_attention_selected_workspace_bytes(cache, selection, heads)))
                binding.dspark_kv4_select(cache, batch, self.bounds[i], turned, selection, work, first=self.first,
                                          last=self.last)
                binding.dspark_kv4_attention_selected(cache, selection, turned, y, t.dim ** -0.5, work)
            else:
                work = self.room(binding.dspark_kv4_attention_workspace_bytes(cache, batch, heads))
                binding.dspark_kv4_attention(cache, batch, turned, y, t.dim ** -0.5, work)
            x = x + y.flatten(1) @ t.out[i]
        return t.norm(x) @ t.head

    def adjust(self, logits, drafts, draft):
        """In place: what a request has said and the drafts before a row count against a token, and no other than the
        allowed ones may come."""
        rows = None if self.mask is None else torch.zeros(logits.shape[0], dtype=torch.int32, device=self.device)
        binding.dspark_logits_adjust(self.said, logits, logits, drafts=drafts, draft=draft, repetition=self.repetition,
                                     presence=self.presence, mask=self.mask, mask_rows=rows)
        return logits

    def prefill(self, prompts):
        sizes = [p.numel() for p in prompts]
        add = torch.tensor(sizes, dtype=torch.int32, device=self.device)
        row_start = torch.nn.functional.pad(torch.cumsum(add, 0), (1, 0)).int()
        self.grow(add)
        if not bool(self.granted.all()):
            self.leave(self.slots)
            raise RuntimeError("the pool has no room for the prompts")
        padded = torch.nn.utils.rnn.pad_sequence(prompts, batch_first=True)
        binding.dspark_tokens_count(self.said, padded, add, prompt=True, reset=True)
        logits = self.forward(torch.cat(prompts), row_start, max(max(sizes), self.drafts + 2))
        last = self.adjust(logits[(row_start[1:] - 1).long()], 0, None).argmax(-1)
        self.count(last[:, None], torch.ones_like(add))
        return last

    def count(self, tokens, count):
        binding.dspark_tokens_count(self.said, tokens, count)

    def verify(self, last, draft, keep=True):
        """One verification, as speculative_step's; the accepted tokens are counted if they are kept."""
        b, p = draft.shape
        rows = torch.empty(b, p + 1, dtype=torch.int64, device=self.device)
        binding.dspark_build_verify_tokens(last, draft, rows, b, draft.stride(0), p)
        before = self.lens.clone()
        self.grow(torch.full((b,), p + 1, dtype=torch.int32, device=self.device))
        row_start = torch.arange(0, b * (p + 1) + 1, p + 1, dtype=torch.int32, device=self.device)
        logits = self.adjust(self.forward(rows.flatten(), row_start, p + 1), p, draft)
        accepted = torch.empty(b, p + 1, dtype=torch.int64, device=self.device)
        count = torch.empty(b, dtype=torch.int32, device=self.device)
        wanted = torch.full((b,), p, dtype=torch.int32, device=self.device)
        binding.dspark_greedy_accept_noalloc(logits, draft, wanted, accepted, count, b, draft.stride(0), p,
                                             logits.shape[1])
        accepted.masked_fill_((self.granted == 0)[:, None], -1)
        count = count * self.granted
        if keep:
            self.count(accepted, count)
        binding.dspark_pages_trim(self.pool, self.slots, before + count)
        return accepted, count

    def compact(self):
        """As speculative_step's; the pages' bounds move with their data."""
        to, src, dst = (torch.empty_like(self.refs) for _ in range(3))
        count = torch.empty(1, dtype=torch.int32, device=self.device)
        binding.dspark_pages_compact(self.pool, self.table, self.refs, to, src, dst, count)
        binding.dspark_pages_copy(self.data, src, dst, count=count)
        binding.dspark_pages_copy(self.bounds, src, dst, count=count)
        return (self.refs > 0).sum()


def main(requests=6, drafts=5, steps=5, vocab=4096, hidden=256, layers=2, kv_heads=2, group=4, dim=64, page_size=16,
         max_tokens=640, agree=0.7, seed=0, device="cuda", longest=500, **kw):
    """Runs `steps` verifications; returns the server, the prompts and the tokens each request got.  A share `agree` of
    the drafts is what the target would say next (the random draft tables seldom agree with it)."""
    g = torch.Generator(device=device).manual_seed(seed)
    target = Target(vocab, hidden, layers, kv_heads, group, dim, device, seed)
    server = Server(target, requests, max_tokens, page_size, requests * max_tokens // page_size, drafts, device, **kw)
    drafter = Drafter(vocab, requests, drafts, device)
    prompts = [torch.randint(0, vocab, (int(n),), device=device, generator=g)
               for n in torch.randint(1, longest, (requests,), generator=torch.Generator().manual_seed(seed))]
    last = server.prefill(prompts)
    got = [last[:, None]]
    for _ in range(steps):
        draft = drafter.draft(last, server.lens)
        for j in range(drafts):
            keep = server.lens.clone()
            accepted, count = server.verify(last, draft, keep=False)
            say = newest(accepted, count, last)
            binding.dspark_pages_trim(server.pool, server.slots, keep)
            here = (count.long() - 1 == j) & (torch.rand(requests, device=device, generator=g) < agree)
            draft[:, j] = torch.where(here, say, draft[:, j])
        accepted, count = server.verify(last, draft)
        last = newest(accepted, count, last)
        got.append(accepted)
    return server, prompts, got


if __name__ == "__main__":
    server, prompts, got = main(presence=0.5, repetition=1.1)
    kept = [(x >= 0).sum(1).tolist() for x in got[1:]]
    print("tokens of each request and step:", kept)
    print("cached tokens:", server.lens.tolist(), "pages a row attends to:", server.top)
    print("tokens said:", server.said.counts.sum(1).tolist())
