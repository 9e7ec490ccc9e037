"""Steps captured with copies, fills and other streams' work in between: the calls' kernels, some of which may begin while
the one before them runs, come behind nodes that are no kernels, and behind two nodes at once."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests.test_gpu_kv4_cache import ints
from tests.test_gpu_kv4_select import Case
from tests.test_gpu_tokens import Table

pytestmark = pytest.mark.gpu


# the launch of one kernel, of clusters, and of three kernels
@pytest.mark.parametrize("kw", [dict(lens=[400, 300]), dict(lens=[16 * 150, 16 * 700]), dict(lens=[400, 300], wide=True)])
@pytest.mark.parametrize("two_graphs", [False, True])
def test_a_step_behind_copies_and_joins(kw, two_graphs):
    c = Case(rows=[2, 1], page=16, heads=2, group=2, dim=64, top=5, last=2, **kw)
    c.bound_all()
    pages, kept = c.select()
    want, want_pages, want_kept = c.attend()[0].clone(), pages.copy(), kept.copy()
    size = max(binding.dspark_kv4_select_workspace_bytes(c.cache, c.batch, c.selection),
               binding.dspark_kv4_attention_selected_workspace_bytes(c.cache, c.selection, 4))
    ws, out = c.scratch(size), torch.empty_like(c.q)
    given, late = c.q.clone(), torch.empty_like(c.q)
    held, data = c.batch.tensors[1].clone(), c.data.clone()

    def choose():
        c.data.copy_(data)                   # a copy, then the bounds
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        binding.dspark_kv4_bound_pages(c.cache, c.batch, c.bounds)
        with torch.cuda.stream(side):
            late.copy_(given)
            c.q.copy_(late)
            c.batch.tensors[1].copy_(held)
        torch.cuda.current_stream().wait_stream(side)  # two nodes, then the selection
        binding.dspark_kv4_select(c.cache, c.batch, c.bounds, c.q, c.selection, ws, first=c.first, last=c.last)

    def attend():
        out.zero_()                          # a fill, then the attention, in the selection's workspace
        binding.dspark_kv4_attention_selected(c.cache, c.selection, c.q, out, c.scale, ws)

    choose()
    attend()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2 if two_graphs else 1)]
    with torch.cuda.graph(graphs[0]):
        choose()
        if not two_graphs:
            attend()
    if two_graphs:
        with torch.cuda.graph(graphs[1]):
            attend()
    for _ in range(3):
        c.q.zero_()
        c.pages.fill_(-9)
        c.kept.fill_(-9)
        out.fill_(-9)
        ws.fill_(0xFF)
        c.data.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(c.pages.cpu().numpy(), want_pages) and np.array_equal(c.kept.cpu().numpy(), want_kept)
        assert torch.equal(out, want)


@pytest.mark.parametrize("width", [0, 300, 20000])
def test_counts_behind_copies(width):
    rng = np.random.default_rng(width)
    t = Table(40, 5000)
    tokens = torch.from_numpy(rng.integers(0, 5000, (40, width))).cuda()
    ids, lens, held = torch.zeros_like(tokens), ints([0] * 40), ints([width] * 40)

    def step():
        t.wide.fill_(7)
        lens.copy_(held)
        ids.copy_(tokens)
        binding.dspark_tokens_count(t.table, ids, lens, reset=True)
        binding.dspark_tokens_count(t.table, ids, lens, prompt=True)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        ids.zero_()
        lens.zero_()
        t.wide_marks.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(40):
            t.want[i] = np.bincount(tokens[i].cpu().numpy(), minlength=5000)
        t.prompt = t.want > 0
        t.check()
