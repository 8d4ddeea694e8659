"""States that hold infinities and NaN: e^g S stays what it is, through
sequences of any length and single tokens."""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import linattn_ref as ref
from tests.test_gpu_linattn import DTYPES, SCALE, dev, host, make

pytestmark = pytest.mark.gpu

INF = float("inf")


def spoiled(state):
    state[:, 0, 3, 5], state[:, 1, 0, 7], state[:, 1, 2, 1] = INF, -INF, float("nan")
    return state


def same(got, want):
    """Infinities and NaN where the definition has them, the rest finite."""
    got = host(got).reshape(want.shape)
    return (np.array_equal(np.isnan(got), np.isnan(want)) and
            np.array_equal(np.isposinf(got), np.isposinf(want)) and
            np.array_equal(np.isneginf(got), np.isneginf(want)))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_empty_sequences_pass_them_on(dtype):
    x = make((0, 4, 0), 2, 2, 2, 8, 16, dtype, 100)
    state = spoiled(x["state"]).cuda()
    args = [x[n].cuda() for n in "qkv"] + [x["g"].cuda()]
    _, last = ps.linattn(*args, SCALE, x["ends"].cuda(), state, want_state=True)
    ds = ps.linattn_grad(x["do"].cuda(), *args, SCALE, x["ends"].cuda(), dstate_out=state, want_dstate=True)[3]
    none = [x[n][:0].view(3, 0, 2, d).cuda() for n, d in (("q", 8), ("k", 8), ("v", 16))]
    _, dense = ps.linattn(*none, args[3], SCALE, state=state, want_state=True)
    bits = lambda t: t.view(torch.int32)  # noqa: E731
    for got in (last, ds):
        assert torch.equal(bits(got[::2].contiguous()), bits(state[::2].contiguous()))
    assert torch.equal(bits(dense), bits(state))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", [(1, 3), (70, 130), (1500, 1300)])
@pytest.mark.parametrize("width", [16, 128])
def test_they_reach_the_last_state(width, lens, dtype):
    x = make(lens, 2, 2, 2, width, width, dtype, 101)
    x["g"] = torch.tensor([-0.013, -0.0021])
    x["state"], x["dlast"] = spoiled(x["state"]), spoiled(x["dlast"])
    names = ("do", "q", "k", "v")
    args = [dev(x, n, lens, True) for n in names]
    g, ends = x["g"].cuda(), x["ends"].cuda()
    out, last = ps.linattn(*args[1:], g, SCALE, ends, x["state"].cuda(), want_state=True)
    h = [host(x[n]) for n in names]
    with np.errstate(invalid="ignore"):
        wout, wlast = ref.forward(*h[1:], x["g"].numpy(), SCALE, lens, host(x["state"]))
        want = ref.backward(*h, x["g"].numpy(), SCALE, lens, host(x["state"]), host(x["dlast"]))
    assert same(last, wlast)
    # an output that adds one up is not finite; others are
    assert np.array_equal(np.isfinite(host(out)), np.isfinite(wout))
    grads = ps.linattn_grad(*args, g, SCALE, ends, x["state"].cuda(), x["dlast"].cuda(), True)
    for a, w in zip(grads[:3], want):
        assert np.array_equal(np.isfinite(host(a)), np.isfinite(w))
    assert same(grads[3], want[3])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("widths", [(16, 16), (128, 128), (17, 9)])
def test_single_tokens_keep_them(widths, dtype):
    dk, dv = widths
    x = make((1,) * 5, 2, 2, 2, dk, dv, dtype, 102)
    x["g"] = torch.tensor([-0.013, -0.0021])
    state = spoiled(x["state"])
    out, new = ps.linattn_step(*[x[n].cuda() for n in "qkv"], x["g"].cuda(), state.cuda(), SCALE)
    with np.errstate(invalid="ignore"):
        wout, wnew = ref.forward(*[host(x[n]) for n in "qkv"], x["g"].numpy(), SCALE, (1,) * 5, host(state))
    assert same(new, wnew) and same(out, wout)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scale", [INF, float("nan")])
def test_a_scale_that_is_not_finite_is_seen(scale, dtype):
    x = make((70,), 2, 2, 2, 16, 16, dtype, 103, state=False)
    args = [x[n].cuda() for n in ("do", "q", "k", "v")] + [torch.tensor([-0.013, 0.0]).cuda()]
    out, _ = ps.linattn(*args[1:], scale, x["ends"].cuda())
    grads = ps.linattn_grad(*args, scale, x["ends"].cuda(), want_dstate=True)
    for t in (out, *grads):
        assert not torch.isfinite(t).any()
