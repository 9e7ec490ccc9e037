"""The example of examples/long_context_step.py: rotated keys, bounds, selections, adjusted logits and token counts as
they are used together.  Whether penalties and masks hold is exact; tokens are compared with one pass over the whole
sequence where the selections hold every page."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("long_context_step", os.path.join(ROOT, "examples",
                                                                                    "long_context_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def said(got, i):
    return torch.cat([x[i][x[i] >= 0] for x in got])


def check_books(server, prompts, got):
    """Lengths, pages and the token table after a run."""
    page = server.pool.struct.page_size
    for i in range(server.requests):
        tokens = said(got, i)
        assert server.lens[i].item() == prompts[i].numel() + tokens.numel() - 1
        vocab = server.said.counts.shape[1]
        assert torch.equal(server.said.counts[i].long(), torch.bincount(tokens, minlength=vocab))
    held = [-(-n // page) for n in server.lens.tolist()]
    assert server.refs.sum().item() == sum(held) and server.refs.max().item() <= 1


@pytest.mark.parametrize("kw", [dict(top=40), dict(top=8, presence=0.3, repetition=1.2),
                                dict(top=5, first=0, last=1, requests=3, drafts=2, page_size=32, dim=128, kv_heads=1,
                                     group=8), dict(top=4, layers=1, page_size=64, drafts=7, agree=1.0)])
def test_example(example, kw):
    server, prompts, got = example.main(steps=3, **kw)
    torch.cuda.synchronize()
    counts = torch.stack([(x >= 0).sum(1) for x in got[1:]])
    assert counts.min() >= 1 and counts.max() <= server.drafts + 1
    check_books(server, prompts, got)


def test_agreeing_drafts_are_accepted(example):
    server, prompts, got = example.main(steps=3, layers=1, top=6, presence=0.2, agree=1.0)
    counts = torch.stack([(x >= 0).sum(1) for x in got[1:]])
    assert counts.max() == server.drafts + 1


def test_a_large_presence_penalty_lets_no_token_come_twice(example):
    server, prompts, got = example.main(steps=4, presence=1e4, agree=1.0)
    check_books(server, prompts, got)
    for i in range(server.requests):
        tokens = said(got, i)
        assert tokens.unique().numel() == tokens.numel()


def test_only_allowed_tokens_come(example):
    allowed = torch.zeros(4096, dtype=torch.bool, device="cuda")
    allowed[5::7] = True
    server, prompts, got = example.main(steps=3, allowed=allowed)
    for i in range(server.requests):
        assert allowed[said(got, i)].all()


def test_selections_of_all_pages_say_what_one_pass_says(example):
    """As the test of speculative_step: logits of about 1 from 4-bit keys and values of rows whose inputs differ in the
    last bits of BF16."""
    server, prompts, got = example.main(steps=4, top=40)
    fresh = example.Server(server.target, server.requests, 640, 16, server.refs.numel(), server.drafts, server.device)
    add = server.lens.clone()
    starts = torch.nn.functional.pad(torch.cumsum(add, 0), (1, 0)).int()
    fresh.grow(add)
    sequences = [torch.cat([prompts[i], said(got, i)]) for i in range(server.requests)]
    logits = fresh.forward(torch.cat([s[:-1] for s in sequences]), starts, int(add.max())).float()
    for i in range(server.requests):
        n0 = prompts[i].numel()
        rows = logits[starts[i] + n0 - 1:starts[i + 1]]
        mine = rows.gather(1, sequences[i][n0:, None])[:, 0]
        assert ((rows.max(1).values - mine) <= 0.35).all()


def test_compaction_moves_bounds_with_the_pages(example):
    server, _, _ = example.main(steps=1)
    lens = server.lens.tolist()
    before = [[server.bounds[layer][server.table[i, :-(-lens[i] // 16)].long()].clone() for i in (0, 2, 4)]
              for layer in range(2)]
    server.leave(server.slots[1::2].contiguous())
    server.compact()
    for layer in range(2):
        for i, want in zip((0, 2, 4), before[layer]):
            assert torch.equal(server.bounds[layer][server.table[i, :want.shape[0]].long()], want)
