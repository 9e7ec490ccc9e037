"""The example of examples/speculative_step.py: what it leaves in the page tables and the cache, and that
verifying in steps of several rows gives the tokens that one pass over the whole sequence gives."""
import importlib.util
import os

import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("speculative_step", os.path.join(ROOT, "examples",
                                                                                   "speculative_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kw", [dict(), dict(requests=3, drafts=1, page_size=32, dim=128, kv_heads=1, group=8, steps=3),
                                dict(requests=5, drafts=7, page_size=64, layers=1, agree=1.0, steps=4)])
def test_example(example, kw):
    server, prompts, got = example.main(**kw)
    torch.cuda.synchronize()
    b, page = server.requests, server.pool.struct.page_size
    counts = torch.stack([(x >= 0).sum(1) for x in got[1:]])
    assert counts.min() >= 1 and counts.max() <= server.drafts + 1
    if kw.get("agree") == 1.0:
        assert counts.max() == server.drafts + 1  # drafts that the target agrees with are accepted
    sequences = []
    for i in range(b):
        tokens = torch.cat([prompts[i]] + [x[i][x[i] >= 0] for x in got])
        # every token but the last is cached
        assert server.lens[i].item() == tokens.numel() - 1
        sequences.append(tokens)
    lens = server.lens.tolist()
    held = [-(-n // page) for n in lens]
    assert server.refs.sum().item() == sum(held) and server.refs.max().item() <= 1
    for i in range(b):
        ids = server.table[i].tolist()
        assert all(p >= 0 for p in ids[:held[i]]) and all(p == -1 for p in ids[held[i]:])
    used = [p for i in range(b) for p in server.table[i].tolist()[:held[i]]]
    assert len(set(used)) == len(used)

    # one pass over the whole sequences: the same cached bytes up to what the steps' BF16 projections round
    # differently, and logits that rank the emitted tokens first or within BF16's resolution of the first
    fresh = example.Server(server.target, b, 400, page, server.refs.numel(), server.drafts, server.device)
    add = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = torch.nn.functional.pad(torch.cumsum(add, 0), (1, 0)).int()
    fresh.grow(add)
    logits = fresh.forward(torch.cat([s[:-1] for s in sequences]), starts, max(lens)).float()
    for i in range(b):
        n0 = prompts[i].numel()
        rows = logits[starts[i] + n0 - 1:starts[i + 1]]
        said = sequences[i][n0:]
        top = rows.max(1).values
        mine = rows.gather(1, said[:, None])[:, 0]
        # logits are of size about 1 and come from 4-bit keys and values of rows whose inputs differ in the last
        # bits of BF16: codes at a rounding boundary may change by a step
        assert ((top - mine) <= 0.35).all(), (top - mine).max()


def test_leaving_compacting_and_forking(example):
    server, _, _ = example.main(requests=6, steps=2)
    lens = server.lens.tolist()
    before = [[server.cached(layer, slot, lens[slot]) for slot in (0, 2, 4)] for layer in range(2)]
    server.leave(server.slots[1::2].contiguous())
    held = sum(-(-lens[s] // 16) for s in (0, 2, 4))
    assert server.compact().item() == held and (server.refs[:held] == 1).all()
    server.fork(server.slots[2:3], server.slots[3:4])
    assert server.lens.tolist() == [lens[0], 0, lens[2], lens[2], lens[4], 0]
    for layer in range(2):
        for slot, want in zip((0, 2, 4), before[layer]):
            got = server.cached(layer, slot, lens[slot])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        fork = server.cached(layer, 3, lens[2])
        assert torch.equal(fork[0], before[layer][1][0]) and torch.equal(fork[1], before[layer][1][1])
    # the branches part: a shared last page is copied for the one that grows
    add = torch.tensor([0, 0, 0, 3, 0, 0], dtype=torch.int32, device="cuda")
    server.grow(add)
    assert server.granted.tolist() == [1] * 6
    partly = lens[2] % 16 != 0
    assert (server.copy_src[3].item() >= 0) == partly
    kept = server.cached(0, 2, lens[2])
    assert torch.equal(kept[0], before[0][1][0])
