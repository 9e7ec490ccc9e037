"""The steps of examples/speculative_step.py where the cache has no room for some requests: these keep their tokens and
get no new ones, the others go on."""
import pytest
import torch

from tests.test_gpu_speculative_example import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_requests_that_have_reached_their_most_tokens(example):  # noqa: F811
    """Tables of 112 tokens, prompts of up to 99: some requests are refused before the others."""
    server, prompts, got = example.main(max_tokens=112, steps=6)
    counts = torch.stack([(x >= 0).sum(1) for x in got[1:]])
    assert counts.min() == 0 and counts.max() >= 1
    lens = server.lens.tolist()
    assert max(lens) <= 112
    sequences = [torch.cat([prompts[i]] + [x[i][x[i] >= 0] for x in got]) for i in range(server.requests)]
    assert lens == [s.numel() - 1 for s in sequences]
    # the same tokens in one pass: what is cached of them in the first layer, whose inputs are the embeddings alone
    fresh = example.Server(server.target, server.requests, 112, 16, server.refs.numel(), server.drafts, server.device)
    add = torch.tensor(lens, dtype=torch.int32, device="cuda")
    fresh.grow(add)
    starts = torch.nn.functional.pad(torch.cumsum(add, 0), (1, 0)).int()
    fresh.forward(torch.cat([s[:-1] for s in sequences]), starts, max(lens))
    for i in range(server.requests):
        for a, b in zip(server.cached(0, i, lens[i]), fresh.cached(0, i, lens[i])):
            # projections of other batch sizes may round to the other side of a code's boundary
            assert ((a - b).abs() > 0.3 * b.abs().clamp(min=0.3)).float().mean() < 0.02, i


def test_a_refused_request_is_left_as_it_was(example):  # noqa: F811
    server, _, _ = example.main(requests=4, steps=1, max_tokens=160)
    lens = server.lens.clone()
    before = [[server.cached(layer, i, n) for i, n in enumerate(lens.tolist())] for layer in range(2)]
    tables = server.table.clone()
    held = server.refs.clone()
    server.refs[server.refs == 0] = 1  # no page is free: requests without room in their last page are refused
    last = torch.zeros(4, dtype=torch.int64, device="cuda")
    draft = torch.ones(4, server.drafts, dtype=torch.int64, device="cuda")
    accepted, count = server.verify(last, draft)
    full = lens % 16 + server.drafts + 1 > 16
    full |= lens % 16 == 0
    assert full.any()
    assert (count[full] == 0).all() and (accepted[full] == -1).all() and (count[~full] >= 1).all()
    assert torch.equal(server.lens, lens + count)
    assert torch.equal(server.table, tables) and torch.equal(server.refs[held > 0], held[held > 0])
    for layer in range(2):
        for i, n in enumerate(lens.tolist()):
            for a, b in zip(server.cached(layer, i, server.lens[i].item()), before[layer][i]):
                assert torch.equal(a[:n], b), (layer, i)


def test_prompts_that_do_not_fit_are_refused(example):  # noqa: F811
    with pytest.raises(RuntimeError, match="room"):
        example.main(requests=3, max_tokens=16, steps=1)
