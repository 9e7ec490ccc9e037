"""Steps captured with copies, fills and other streams' work in between: the calls' kernels, some of which may begin while
the one before them runs, come behind nodes that are no kernels, and behind two nodes at once."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests.test_gpu_kv4_cache import ints
from tests.test_gpu_kv4_select import Case
from tests.test_gpu_tokens import Table

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def test_first_calls_captured():
    """A process whose first call of every entry point is a captured one."""
    code = """
import sys
sys.path.insert(0, %r)
import torch
from dspark_markov_draft_anchor_gb300 import binding as b
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
page, heads, dim, n = 16, 2, 64, 16 * 2100 + 5
ids = torch.randperm(2101, generator=torch.Generator().manual_seed(0)).int().cuda()[None]
z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")
def step(top, width, wide):
    cache = b.Kv4Cache(z(2101, b.kv4_page_bytes(page, heads, dim), t=torch.uint8), page, heads, dim)
    table = ids[:, :width].contiguous()
    lens = ints([min(n, 16 * width)])
    batch = b.Kv4Batch(ints([0, 3]), lens, table, total_rows=3, max_rows=3)
    rot = b.Kv4Rotation(z(n, 32, t=torch.float32) + 1, z(n, 32, t=torch.float32))
    bounds = z(2101, b.kv4_bounds_bytes(heads, dim), t=torch.uint8)
    sel = b.Kv4Selection(z(3, heads, top, t=torch.int32), z(3, t=torch.int32))
    ws = z(max(b.dspark_kv4_select_workspace_bytes(cache, batch, sel),
               b.dspark_kv4_attention_selected_workspace_bytes(cache, sel, 4)), t=torch.uint8)
    k, q, out = z(3, heads, dim) + 2, z(3, 4, dim) + 1, z(3, 4, dim)
    said = b.TokenTable(z(40, 5000, t=torch.int32), z(40, 2, 157, t=torch.int32))
    tokens, held = z(40, wide, t=torch.int64), ints([wide] * 40)
    logits = z(40, 5000)
    pen = z(40, t=torch.float32) + 2
    def run():
        b.dspark_kv4_append_rotated(cache, batch, rot, k, k, q, q)
        b.dspark_kv4_bound_pages(cache, batch, bounds)
        b.dspark_kv4_select(cache, batch, bounds, q, sel, ws)
        b.dspark_kv4_attention_selected(cache, sel, q, out, 0.1, ws)
        b.dspark_tokens_count(said, tokens, held, reset=True)
        b.dspark_logits_adjust(said, logits, logits, presence=pen)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    torch.cuda.synchronize()
    assert sel.lens.tolist()[2] == (min(len(ids[0]), top, width) - 1) * page + (5 if width == 2101 else 16), sel.lens
    assert out.float().abs().max() > 0 and said.counts[:, 0].tolist() == [wide] * 40
    assert logits[:, 0].tolist() == [-2.0] * 40 and not logits[:, 1:].any()
for args in ((64, 2101, 20000), (64, 400, 3), (4, 100, 3), (64, 50, 3)):
    step(*args)
print("well")
""" % ROOT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "well", r.stdout + r.stderr


@pytest.mark.parametrize("graphs", [False, True])
def test_two_steps_at_once(graphs):
    """Two streams, each with its own cache, selection and workspace."""
    cases = [Case(rows=[2, 1], lens=[16 * 900, 300], page=16, heads=2, group=2, dim=64, top=5, last=2, seed=s, wide=s == 1)
             for s in (0, 1)]
    steps, wants = [], []
    for c in cases:
        c.bound_all()
        pages, kept = c.select()
        wants.append((pages.copy(), kept.copy(), c.attend()[0].clone()))
        size = max(binding.dspark_kv4_select_workspace_bytes(c.cache, c.batch, c.selection),
                   binding.dspark_kv4_attention_selected_workspace_bytes(c.cache, c.selection, 4))
        ws, out = c.scratch(size), torch.zeros_like(c.q)

        def step(c=c, ws=ws, out=out):
            for _ in range(20):
                binding.dspark_kv4_bound_pages(c.cache, c.batch, c.bounds)
                binding.dspark_kv4_select(c.cache, c.batch, c.bounds, c.q, c.selection, ws, first=c.first, last=c.last)
                binding.dspark_kv4_attention_selected(c.cache, c.selection, c.q, out, c.scale, ws)
        c.pages.fill_(-9)
        c.kept.fill_(-9)
        steps.append((step, out))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    runs = []
    for (step, _), s in zip(steps, streams):
        if graphs:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
            runs.append(graph.replay)
        else:
            runs.append(step)
    torch.cuda.synchronize()
    for run, s in zip(runs, streams):
        with torch.cuda.stream(s):
            run()
    torch.cuda.synchronize()
    for c, (_, out), (pages, kept, want) in zip(cases, steps, wants):
        assert np.array_equal(c.pages.cpu().numpy(), pages) and np.array_equal(c.kept.cpu().numpy(), kept)
        assert torch.equal(out, want)
