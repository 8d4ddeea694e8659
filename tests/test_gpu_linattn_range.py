"""Linear attention on the GPU where rows of very different sizes lie in one
chunk: a large value changes no token that does not see it, and ordinary ones
stay within the tolerances of test_gpu_linattn."""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import linattn_ref as ref
from tests.test_gpu_linattn import DTYPES, SCALE, dev, host, make, near

pytestmark = pytest.mark.gpu

LARGE = 6e4                       # near f16's end


def run(x, lens, grad=False, scale=SCALE):
    names = ("do", "q", "k", "v") if grad else ("q", "k", "v")
    args = [dev(x, n, lens, True) for n in names]
    g, ends = x["g"].cuda(), x["ends"].cuda()
    state = None if x["state"] is None else x["state"].cuda()
    if not grad:
        return ps.linattn(*args, g, scale, ends, state, want_state=True)
    dlast = None if x["dlast"] is None else x["dlast"].cuda()
    return ps.linattn_grad(*args, g, scale, ends, state, dlast, True)


def definition(x, lens, grad=False, scale=SCALE, absolute=False):
    f = (lambda t: None if t is None else np.abs(host(t))) if absolute else host
    if not grad:
        return ref.forward(f(x["q"]), f(x["k"]), f(x["v"]), x["g"].numpy(), scale, lens, f(x["state"]))
    return ref.backward(*[f(x[n]) for n in ("do", "q", "k", "v")], x["g"].numpy(), scale, lens, f(x["state"]),
                        f(x["dlast"]))


def held(x, lens, dtype, grad=False, scale=SCALE, skip=()):
    got, want, size = run(x, lens, grad, scale), definition(x, lens, grad, scale), definition(x, lens, grad, scale, True)
    terms = max(lens) + x["q"].shape[-1] + x["v"].shape[-1] + x["g"].numel()
    names = ("dq", "dk", "dv", "dstate") if grad else ("out", "state")
    for a, w, s, name in zip(got, want, size, names):
        if name not in skip:
            near(a, w, s, dtype, terms, name, state=name in ("state", "dstate"))
    return got


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("large", [1e3, 1e4, LARGE])
@pytest.mark.parametrize("width", [64, 128])
def test_a_large_row_changes_no_token_before_it(width, large, dtype):
    lens = (64,)
    x = make(lens, 2, 2, 2, width, width, dtype, 90)
    x["g"] = torch.tensor([-0.01, 0.0])
    clean = run(x, lens)[0]
    x["q"][50, :, 3] = large
    x["k"][55, :, 7] = large
    # outputs past f16's end are not asked for
    scale = SCALE if dtype != "fp16" else 2.0 ** -24
    out = run(x, lens)[0]
    assert torch.equal(out[:50], clean[:50]) and torch.equal(out[51:55], clean[51:55])
    held(x, lens, dtype, scale=scale)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_a_large_row_changes_no_gradient_that_does_not_see_it(dtype):
    lens = (60, 70)
    x = make(lens, 2, 2, 2, 64, 96, dtype, 91)
    x["g"] = torch.tensor([-0.05, 0.0])
    clean = run(x, lens, True)
    for name, at in (("do", 20), ("q", 85), ("k", 30), ("v", 100)):
        y = dict(x)
        y[name] = x[name].clone()
        y[name][at, :, 5] = LARGE
        got = run(y, lens, True)
        end = 60 if at < 60 else 130
        sees = {"dq": range(at, end), "dk": range(60 if at >= 60 else 0, at + 1)}
        sees["dv"] = sees["dk"]
        for a, b, n in zip(got, clean, ("dq", "dk", "dv")):
            other = torch.ones(130, dtype=torch.bool)
            other[list(sees[n])] = False
            assert torch.equal(a[other.cuda()], b[other.cuda()]), (name, n)
    y = dict(x)
    for name, at in (("do", 20), ("q", 85), ("k", 30), ("v", 100)):
        y[name] = x[name].clone()
        y[name][at, :, 5] = LARGE
    y["dlast"] = None                  # times the large k and v it is past f16, whatever the scale
    held(y, lens, dtype, True, 2.0 ** -26 if dtype == "fp16" else SCALE)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("masked", ["k", "v"])
@pytest.mark.parametrize("g", [-0.25, -0.5, -1.0])
def test_a_state_fades_under_masked_tokens(g, masked, dtype):
    # Keys or values of zero after the first ten tokens: what is left of the
    # state is far below the rows, and as exact as ever.
    lens = (64, 130, 11)
    x = make(lens, 2, 2, 2, 64, 64, dtype, 92, state=False)
    x["g"] = torch.tensor([g, g / 2])
    at = 0
    for n in lens:
        x[masked][at + 10:at + n] = 0.0
        at += n
    # outputs of f16 would be below its least numbers: the state alone
    held(x, lens, dtype, skip=("out",) if dtype == "fp16" else ())


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_sizes_change_along_a_sequence(dtype):
    # Rows, and so the state, go from large to small and back; some chunks
    # hold both.
    lens = (400, 0, 300)
    x = make(lens, 2, 2, 2, 64, 128, dtype, 93)
    x["g"] = torch.tensor([-0.02, -0.3])
    size = torch.ones(700)
    size[70:130], size[200:330], size[400:420] = 2.0 ** 8, 2.0 ** -9, 2.0 ** -5
    for n in "kv":
        x[n] = (x[n].float() * size[:, None, None]).to(DTYPES[dtype])
    x["state"] = x["state"] * torch.tensor([2.0 ** 14, 1.0, 2.0 ** -14])[:, None, None, None]
    held(x, lens, dtype, scale=2.0 ** -12)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_a_large_state_over_empty_rows(dtype):
    # States far past f16, and rows of zeros: the state is only decayed.
    lens = (130, 20)
    x = make(lens, 2, 2, 2, 64, 64, dtype, 94)
    x["g"] = torch.tensor([-0.01, 0.0])
    x["state"] = x["state"] * 1e30
    x["k"][:] = 0.0
    held(x, lens, dtype, scale=2.0 ** -100 if dtype != "bf16" else SCALE)
