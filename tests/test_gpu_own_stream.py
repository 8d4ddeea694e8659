"""Tensors that a call makes belong to the stream that it runs on: memory that
another stream's pending work may still use is not written."""
import pytest
import torch

import prefix_scan_amd as ps

pytestmark = pytest.mark.gpu

T, H, D = 3001, 4, 64


def calls():
    x = torch.randn(1, T, H, D, device="cuda")
    g = torch.full((H,), -0.1, device="cuda")
    packed, ends = x[0], torch.tensor([1000, T - 7], dtype=torch.int32, device="cuda")
    state = torch.randn(T, H, 8, D, device="cuda")
    after = torch.empty_like(state)
    narrow = x[0, ..., :8].contiguous()
    logits, u = torch.randn(50000, 16, device="cuda"), torch.rand(50000, device="cuda")
    return {
        "linattn": lambda s: [ps.linattn(x, x, x, g, stream=s)[0]],
        "packed": lambda s: [ps.linattn(packed, packed, packed, g, ends=ends, stream=s)[0]],
        "states": lambda s: [ps.linattn(x, x, x, g, want_state=True, stream=s)[1]],
        "linattn_grad": lambda s: [t for t in ps.linattn_grad(x, x, x, x, g, stream=s)[:3]],
        "packed_grad": lambda s: [t for t in ps.linattn_grad(packed, packed, packed, packed, g, ends=ends,
                                                             dk=torch.empty_like(packed), stream=s)[::2]],
        "linattn_step": lambda s: [ps.linattn_step(narrow, narrow, packed, g, state, state_out=after, stream=s)[0]],
        "sample_logits": lambda s: list(ps.sample_logits(logits, u, stream=s)),
    }


@pytest.mark.parametrize("name", ["linattn", "packed", "states", "linattn_grad", "packed_grad", "linattn_step",
                                  "sample_logits"])
def test_new_tensors_come_from_the_streams_memory(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = [t.clone() for t in call(None)]
    call(side)                                   # scratch is there
    torch.cuda.synchronize()
    shapes = [(t.shape, t.dtype) for t in want]
    with torch.cuda.stream(side):
        mine = [torch.empty(s, dtype=d, device="cuda") for s, d in shapes]
    at = {t.data_ptr() for t in mine}
    del mine
    got = call(side)
    torch.cuda.synchronize()
    assert {t.data_ptr() for t in got} <= at
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def word_calls():
    n = 300007
    x = torch.randint(0, 9, (n,), dtype=torch.int32, device="cuda")
    ends = torch.cumsum(x, 0).to(torch.int32)
    flags = (x == 0).to(torch.int32)
    return {
        "runs_layout": lambda s: [ps.runs_layout_u32(x, want_entries=False, stream=s)[0]],
        "runs_owner": lambda s: [ps.runs_owner_u32(ends, x, stream=s)],
        "runs_owner_all": lambda s: [ps.runs_owner_all_u32(ends, n, stream=s)],
        "segscan": lambda s: list(ps.segscan_u32(x, 7, stream=s)),
        "segscan_flags": lambda s: list(ps.segscan_flags_u32(x, flags, stream=s)[:2]),
        "compact": lambda s: [ps.compact_flags_u32(flags, want_count=False, stream=s)[0]],
        "radix": lambda s: [ps.radix_perm_u32(x, 4, stream=s)],
    }


@pytest.mark.parametrize("name", ["runs_layout", "runs_owner", "runs_owner_all", "segscan", "segscan_flags",
                                  "compact", "radix"])
def test_so_do_those_of_the_primitives(name):
    call = word_calls()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = [t.clone() for t in call(None)]
    call(side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        mine = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (300007, 300007)]
    at = {t.data_ptr() for t in mine}
    del mine
    got = call(side)
    torch.cuda.synchronize()
    assert got[0].data_ptr() in at
    for a, b in zip(got, want):
        assert torch.equal(a, b)
