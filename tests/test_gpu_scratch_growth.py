"""Scratch buffers on the GPU: one that a captured graph holds outlives a
larger one that takes its place, others are given back."""
import gc
import weakref

import pytest
import torch

import prefix_scan_amd as ps

pytestmark = pytest.mark.gpu


def held(stream):
    return weakref.ref(ps._scratch[(0, stream.cuda_stream)].buf)


def test_growing_keeps_what_a_graph_holds():
    stream = torch.cuda.Stream()
    sort = lambda t: ps.radix_perm_u32(t, 4, stream=stream)  # noqa: E731
    small, large = (torch.randint(0, 1 << 30, (n,), dtype=torch.int32, device="cuda") for n in (5000, 200000))
    x, u = torch.randn(9, 5000, device="cuda"), torch.rand(9, device="cuda")
    out = torch.empty(9, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    sort(small)
    torch.cuda.synchronize()
    first = held(stream)
    sort(large)
    torch.cuda.synchronize()
    gc.collect()
    assert first() is None                      # no graph has seen it
    second = held(stream)
    with torch.cuda.stream(stream):
        ps.sample_logits(x, u, top_k=40, tokens=out)
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ps.sample_logits(x, u, top_k=40, tokens=out)
    sort(torch.randint(0, 1 << 30, (3000000,), dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    gc.collect()
    assert second() is not None and held(stream)() is not second()
    for _ in range(3):
        out.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        sort(large)
        torch.cuda.synchronize()
