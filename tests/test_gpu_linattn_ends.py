"""Lists of ends that are no packed batch: what the header promises of them.
Ends past the rows are cut to them; ends that fall leave outputs and states
unspecified, and touch nothing else."""
import pytest
import torch

import prefix_scan_amd as ps
from tests.test_gpu_linattn import DTYPES, SCALE, decays

pytestmark = pytest.mark.gpu


def guarded(shape, dtype, fill=9.0, edge=4096):
    n = 1
    for s in shape:
        n *= s
    flat = torch.full((n + 2 * edge,), fill, dtype=dtype, device="cuda")
    return flat, flat[edge:edge + n].view(shape)


def untouched(flat, view, fill=9.0):
    edge = (flat.numel() - view.numel()) // 2
    return bool((flat[:edge] == fill).all() and (flat[-edge:] == fill).all())


def inputs(tokens, heads, dk, dv, dtype, seqs):
    gen = torch.Generator().manual_seed(90)
    mk = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    rows = [mk(tokens, heads, d).to(DTYPES[dtype]).cuda() for d in (dv, dk, dk, dv)]
    states = [mk(seqs, heads, dk, dv).cuda() for _ in range(2)]
    return rows, states, torch.from_numpy(decays(heads)).cuda()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens", [90, 1500])
def test_ends_past_the_rows_are_cut(tokens, dtype):
    heads, dk, dv = 2, 40, 64
    (do, q, k, v), (state, dlast), g = inputs(tokens, heads, dk, dv, dtype, 4)
    listed = lambda *e: torch.tensor([x - (1 << 32) if x >= 1 << 31 else x for x in e], dtype=torch.int32).cuda()  # noqa: E731
    for far in (tokens + 1, 1 << 31, (1 << 32) - 1):
        want = ps.linattn(q, k, v, g, SCALE, listed(7, 20, tokens, tokens), state, want_state=True)
        got = ps.linattn(q, k, v, g, SCALE, listed(7, 20, far, far), state, want_state=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = ps.linattn_grad(do, q, k, v, g, SCALE, listed(7, 20, tokens, tokens), state, dlast, True)
        got = ps.linattn_grad(do, q, k, v, g, SCALE, listed(7, 20, far, far), state, dlast, True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens", [90, 2000])
def test_ends_that_fall_touch_nothing_else(tokens, dtype):
    heads, dk, dv = 2, 40, 64
    for ends in ((tokens, 0, tokens, 0, tokens), (tokens, 30, 10), (50, 20, 60, 70, 5, 1 << 30), (-1, 3)):
        (do, q, k, v), (state, dlast), g = inputs(tokens, heads, dk, dv, dtype, len(ends))
        e = torch.tensor(ends, dtype=torch.int32).cuda()
        outs = [guarded(t.shape, t.dtype) for t in (v, q, k, v)]
        last = [guarded(state.shape, torch.float32) for _ in range(2)]
        ps.linattn(q, k, v, g, SCALE, e, state, out=outs[0][1], state_out=last[0][1])
        ps.linattn_grad(do, q, k, v, g, SCALE, e, state, dlast, dq=outs[1][1], dk=outs[2][1], dv=outs[3][1],
                        dstate=last[1][1])
        torch.cuda.synchronize()
        assert all(untouched(*t) for t in outs + last), ends
