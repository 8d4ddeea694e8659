"""Linear attention on the GPU: paths by length, outputs asked for and scale,
within the tolerances of test_gpu_linattn."""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import linattn_ref as ref
from tests.test_gpu_linattn import (DTYPES, HALF, SCALE, check_backward, check_forward, decays, dev, host,
                                    make, near)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", [(1,), (65, 65), (700,), (3000,)])
def test_outputs_alone(lens, dtype):
    # No state is asked for: the state is summed for the outputs alone.
    heads, dk, dv = 3, 72, 128
    x = make(lens, heads, heads, heads, dk, dv, dtype, 21, packed=False, state=False)
    args = [dev(x, n, lens, False) for n in "qkv"]
    g = x["g"].cuda()
    out, none = ps.linattn(*args, g, scale=SCALE)
    assert none is None
    want, _ = ref.forward(*[host(x[n]) for n in "qkv"], x["g"].numpy(), SCALE, lens)
    size, _ = ref.forward(*[np.abs(host(x[n])) for n in "qkv"], x["g"].numpy(), SCALE, lens)
    near(out, want, size, dtype, max(lens) + dk + dv, "out")
    got = ps.linattn_grad(dev(x, "do", lens, False), *args, g, scale=SCALE)
    assert got[3] is None
    names = ("do", "q", "k", "v")
    want = ref.backward(*[host(x[n]) for n in names], x["g"].numpy(), SCALE, lens)
    size = ref.backward(*[np.abs(host(x[n])) for n in names], x["g"].numpy(), SCALE, lens)
    for i, name in enumerate(("dq", "dk", "dv")):
        near(got[i], want[i], size[i], dtype, max(lens) + dk + dv + heads, name)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("width", [64, 128])
def test_many_segments(width, dtype):
    # Few heads and long sequences: so many segments that their states are
    # joined before the sweep.
    check_forward((3000,), 2, 1, 2, width, width, dtype, packed=False, seed=22)
    check_backward((2900,), 1, 1, 1, width, width, dtype, packed=False, seed=23)
    check_backward((0, 2100, 5, 1100), 2, 2, 1, width, width, dtype, seed=24)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("size", [2.0 ** -9, 2.0 ** 5])
def test_magnitudes(size, dtype):
    # Rows far from 1, so that products and states leave f16's range.
    lens, heads, dk, dv = (150, 0, 90), 3, 64, 96
    x = make(lens, heads, heads, heads, dk, dv, dtype, 25)
    for n in "kv":
        x[n] = x[n] * size
        x[n][70:75] = x[n][70:75] * 2.0 ** -3
    x["state"], x["dlast"] = x["state"] * size ** 2, None
    scale = 2.0 ** -10 / size if size > 1 else 16.0
    args = [dev(x, n, lens, True) for n in "qkv"]
    g, ends = x["g"].cuda(), x["ends"].cuda()
    out, last = ps.linattn(*args, g, scale=scale, ends=ends, state=x["state"].cuda(), want_state=True)
    h = [host(x[n]) for n in "qkv"]
    want, wlast = ref.forward(*h, x["g"].numpy(), scale, lens, host(x["state"]))
    big, blast = ref.forward(*[np.abs(t) for t in h], x["g"].numpy(), scale, lens, np.abs(host(x["state"])))
    terms = max(lens) + dk + dv
    near(out, want, big, dtype, terms, "out")
    near(last, wlast, blast, dtype, terms, "state", state=True)


def test_layouts_in_turn():
    # One shape in other strides and types, again
    # and again: each call is answered by its own layout.
    lens, heads, d = (40, 40), 2, 64
    for turn in range(3):
        for dtype in DTYPES:
            x = make(lens, heads, heads, heads, d, d, dtype, 30 + turn, packed=False, state=False)
            dense = [dev(x, n, lens, False) for n in "qkv"]
            want, _ = ref.forward(*[host(x[n]) for n in "qkv"], x["g"].numpy(), SCALE, lens)
            size, _ = ref.forward(*[np.abs(host(x[n])) for n in "qkv"], x["g"].numpy(), SCALE, lens)
            turned = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in dense]
            wide = [torch.cat([t, t], 3)[..., :d] for t in dense]
            for args in (dense, turned, wide, [dense[0], turned[1], wide[2]]):
                out, _ = ps.linattn(*args, x["g"].cuda(), scale=SCALE)
                near(out, want, size, dtype, 40 + 2 * d, "out")
    bad = dense[1].cpu()
    with pytest.raises((TypeError, ValueError)):
        ps.linattn(dense[0], bad, dense[2], x["g"].cuda())
    with pytest.raises((TypeError, ValueError)):
        ps.linattn(dense[0], dense[1].half(), dense[2], x["g"].cuda())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_half_types_are_as_near_as_their_rounding(dtype):
    # The mean error, over the tolerance that a single rounding of the
    # output would have: bf16 also rounds scores and state once each.
    lens, heads, d = (512,), 2, 128
    x = make(lens, heads, heads, heads, d, d, dtype, 40, packed=False, state=False)
    x["g"] = torch.from_numpy(decays(heads))
    out, _ = ps.linattn(*[dev(x, n, lens, False) for n in "qkv"], x["g"].cuda(), scale=SCALE)
    want, _ = ref.forward(*[host(x[n]) for n in "qkv"], x["g"].numpy(), SCALE, lens)
    off = host(out).reshape(want.shape) - want
    # Root mean squares: a rounding to nearest is at most h of its value; the
    # sums' terms are rounded with either sign, so their squares add, to at
    # most h of the outputs' own root mean square for each of the two.
    rms = lambda t: float(np.sqrt((t * t).mean()))  # noqa: E731
    assert rms(off) <= (3.0 if dtype == "bf16" else 1.0) * HALF[dtype] * rms(want) + 2.0 ** -25
