"""Linear attention over packed batches of many sequences, of which few are
cut into segments: every sequence is found, and joined from its own segments.
Tolerances as in test_gpu_linattn."""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests.test_gpu_linattn import DTYPES, SCALE, check_backward, check_forward, decays

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_some_of_many_are_cut(dtype):
    rng = np.random.default_rng(80)
    lens = rng.integers(0, 9, 300)
    lens[[3, 4, 170, 299]] = 1300, 517, 2600, 700      # more than a segment each, next to each other and last
    lens[[5, 171]] = 256, 0
    check_forward(tuple(lens), 2, 2, 1, 64, 48, dtype, seed=81)
    check_backward(tuple(lens), 2, 1, 2, 32, 64, dtype, seed=82)


def test_each_sequence_is_its_own():
    # Thousands of sequences, among them long ones, against each alone.
    gen = torch.Generator().manual_seed(83)
    lens = torch.randint(0, 12, (9000,), generator=gen)
    lens[::1500] = 1500
    lens[8999] = 2000
    heads, dk, dv, n = 4, 64, 64, int(lens.sum())
    mk = lambda *s: torch.randn(s, generator=gen).bfloat16().cuda()  # noqa: E731
    q, k, v = mk(n, heads, dk), mk(n, heads, dk), mk(n, heads, dv)
    g = torch.from_numpy(decays(heads)).cuda()
    ends = torch.cumsum(lens, 0).to(torch.int32).cuda()
    state = torch.randn((9000, heads, dk, dv), generator=gen).cuda()
    out, last = ps.linattn(q, k, v, g, SCALE, ends, state, want_state=True)
    at = [0] + ends.tolist()
    for s in list(range(0, 9000, 1500)) + [8999, 1, 2, 77, 4501, 8998]:
        lo, hi = at[s], at[s + 1]
        a, b = ps.linattn(*[t[lo:hi].contiguous()[None] for t in (q, k, v)], g, SCALE,
                          state=state[s:s + 1], want_state=True)
        # other segments: 32-bit sums in another order, then one bf16 rounding
        assert torch.allclose(out[lo:hi].float(), a[0].float(), rtol=2.0 ** -7, atol=2.0 ** -6 * 30), s
        assert torch.allclose(last[s:s + 1], b, rtol=2.0 ** -12, atol=2.0 ** -10), s
    empty = (lens == 0).cuda()
    assert torch.equal(last[empty], state[empty])
