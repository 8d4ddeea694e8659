"""Packed batches with rows past the last sequence, as a fixed shape leaves
them: nothing there is read, and nothing there is written."""
import pytest
import torch

import prefix_scan_amd as ps
from tests.test_gpu_linattn import DTYPES, SCALE, decays

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shared", [(4, 4, 4), (2, 1, 2), (1, 2, 4), (4, 4, 1)])
def test_gradients_past_the_last_sequence_are_left_alone(shared, dtype):
    heads, tokens, dk, dv = 4, 190, 24, 40
    lens = (40, 0, 75)
    last = sum(lens)
    gen = torch.Generator().manual_seed(70)
    mk = lambda *s: torch.randn(s, generator=gen).to(DTYPES[dtype]).cuda()  # noqa: E731
    do, q, k, v = (mk(tokens, h, d) for h, d in zip((heads,) + shared, (dv, dk, dk, dv)))
    g = torch.from_numpy(decays(heads)).cuda()
    ends = torch.tensor([40, 40, 115], dtype=torch.int32).cuda()
    want = ps.linattn_grad(*[t[:last].contiguous() for t in (do, q, k, v)], g, SCALE, ends)
    # what an earlier call leaves in the scratch
    huge = [torch.full_like(t, float("inf")) for t in (do, q, k, v)]
    ps.linattn_grad(*huge, g, SCALE, torch.tensor([tokens], dtype=torch.int32).cuda())
    for t in (do, q, k, v):
        t[last:] = float("nan")
    outs = [torch.full_like(t, 9.0) for t in (q, k, v)]
    ps.linattn_grad(do, q, k, v, g, SCALE, ends, dq=outs[0], dk=outs[1], dv=outs[2])
    for a, b in zip(outs, want):
        assert (a[last:] == 9).all()
        assert torch.equal(a[:last], b)
