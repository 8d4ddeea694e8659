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


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", [(40, 0, 75), (), (190,), (0, 0)])
def test_tensors_the_call_makes_hold_zeros_there(lens, dtype):
    # What memory held before would reach a model's weights through them.
    heads, tokens, dk, dv = 4, 190, 24, 40
    gen = torch.Generator().manual_seed(71)
    mk = lambda *s: torch.randn(s, generator=gen).to(DTYPES[dtype]).cuda()  # noqa: E731
    do, q, k, v = mk(tokens, heads, dv), mk(tokens, 2, dk), mk(tokens, heads, dk), mk(tokens, 1, dv)
    g = torch.from_numpy(decays(heads)).cuda()
    ends = torch.tensor(lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    last = sum(lens)
    for _ in range(2):
        # memory that the outputs may get
        junk = [torch.full_like(t, float("nan")) for t in (do, q, k, v) for _ in range(3)]
        del junk
        out, _ = ps.linattn(q, k, v, g, SCALE, ends)
        grads = ps.linattn_grad(do, q, k, v, g, SCALE, ends)[:3]
        for t in (out, *grads):
            assert not t[last:].any() and t[:last].isfinite().all()
    if last:
        want, _ = ps.linattn(*[t[:last].contiguous() for t in (q, k, v)], g, SCALE, ends)
        assert torch.equal(out[:last], want)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_given_gradients_stay_as_they_are_beside_new_ones(dtype):
    heads, tokens, d = 4, 150, 24
    gen = torch.Generator().manual_seed(72)
    mk = lambda h: torch.randn((tokens, h, d), generator=gen).to(DTYPES[dtype]).cuda()  # noqa: E731
    do, q, k, v = mk(heads), mk(heads), mk(2), mk(1)
    g = torch.from_numpy(decays(heads)).cuda()
    ends = torch.tensor([70, 110], dtype=torch.int32).cuda()
    want = ps.linattn_grad(do, q, k, v, g, SCALE, ends)
    for mine in range(3):
        given = [torch.full_like(t, 9.0) if i == mine else None for i, t in enumerate((q, k, v))]
        got = ps.linattn_grad(do, q, k, v, g, SCALE, ends, dq=given[0], dk=given[1], dv=given[2])
        for i in range(3):
            assert torch.equal(got[i][:110], want[i][:110])
            assert (got[i][110:] == (9 if i == mine else 0)).all()
