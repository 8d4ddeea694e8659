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
