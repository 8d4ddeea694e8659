"""Single tokens on the GPU over pools of states larger than the caches hold."""
import pytest
import torch

import prefix_scan_amd as ps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("widths", [(128, 128), (100, 120), (90, 121)])
@pytest.mark.parametrize("in_place", [True, False])
def test_a_large_pool(widths, in_place):
    # The definition in float64 on the device, in parts of the rows.  32-bit
    # sums of dk terms, and the output's own bf16 rounding.
    dk, dv = widths
    rows, heads, pool = 210, 33, 230
    gen = torch.Generator(device="cuda").manual_seed(50)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = (randn(rows, heads, d).bfloat16() for d in (dk, dk, dv))
    g = -torch.arange(heads, device="cuda") / 40.0
    state = randn(pool, heads, dk, dv)
    slots = torch.randperm(pool, generator=gen, device="cuda")[:rows].to(torch.int32)
    slots[7] = -1
    before = state.clone()
    to = state if in_place else torch.full_like(state, 5.0)
    out, got = ps.linattn_step(q, k, v, g, state, 0.5, slots, state_out=to)
    assert got is to
    rest = torch.ones(pool, dtype=torch.bool, device="cuda")
    rest[slots[slots >= 0].long()] = False
    assert torch.equal(to[rest], before[rest] if in_place else torch.full_like(to[rest], 5.0))
    assert not out[7].any()
    e = g.double().exp()[:, None, None]
    for r in range(rows):
        if r == 7:
            continue
        s = before[int(slots[r])].double()
        kv = k[r].double()[:, :, None] * v[r].double()[:, None, :]
        want, size = e * s + kv, e * s.abs() + kv.abs()
        assert bool(((to[int(slots[r])] - want).abs() <= 4 * 2.0 ** -23 * size).all()), r
        o = 0.5 * (q[r].double()[:, :, None] * want).sum(1)
        osize = 0.5 * (q[r].double().abs()[:, :, None] * size).sum(1)
        off = (out[r].double() - o).abs()
        assert bool((off <= 2.0 ** -8 * o.abs() + (dk + 8) * 2.0 ** -23 * osize).all()), r
