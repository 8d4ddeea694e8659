"""Linear attention of 16-bit rows on the GPU: nothing but the output's own
rounding may be seen.  Scores and states are multiplied in two parts of 16
bits: bf16's first is cut (what it leaves is below 2^-7 of the number) and its
second rounded (2^-8 of that), 2^-15 of the number; a state that is only read
sums rows in two parts as well, another 2^-15.  f16's are within 2^-15 too.
With A the same sums over absolute values, an output may be off by
    h |out| + 2^-14 A + (tokens + widths + 128) 2^-23 A        h = eps / 2."""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import linattn_ref as ref
from tests.test_gpu_linattn import DTYPES, HALF, decays, dev, host, make

pytestmark = pytest.mark.gpu


def close(got, want, size, dtype, terms, what):
    got = host(got).reshape(want.shape)
    assert np.isfinite(got).all(), what
    tol = HALF[dtype] * np.abs(want) + (2.0 ** -14 + (terms + 128) * 2.0 ** -23) * size + 2.0 ** -25
    off = np.abs(got - want)
    assert (off <= tol).all(), "%s: off by %g where %g is allowed" % (
        what, off.flat[np.argmax(off - tol)], tol.flat[np.argmax(off - tol)])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens", [1, 2, 5])
@pytest.mark.parametrize("widths", [(1, 8), (2, 64), (3, 72)])
def test_products_are_rounded_once(widths, tokens, dtype):
    # Few terms: the rounding of each would show in the sum.
    dk, dv = widths
    lens, heads = (tokens,) * 24, 8
    for state in (True, False):
        x = make(lens, heads, heads, heads, dk, dv, dtype, 60 + tokens, packed=False, state=state)
        names = ("do", "q", "k", "v")
        args = [dev(x, n, lens, False) for n in names]
        g = x["g"].cuda()
        h = [host(x[n]) for n in names]
        a = [np.abs(t) for t in h]
        s, ds = host(x["state"]), host(x["dlast"])
        mag = lambda t: None if t is None else np.abs(t)  # noqa: E731
        put = lambda t: None if t is None else t.cuda()  # noqa: E731
        out, _ = ps.linattn(*args[1:], g, state=put(x["state"]))
        want, _ = ref.forward(*h[1:], x["g"].numpy(), 1.0, lens, s)
        size, _ = ref.forward(*a[1:], x["g"].numpy(), 1.0, lens, mag(s))
        close(out, want, size, dtype, tokens + dk + dv, "out")
        got = ps.linattn_grad(*args, g, state=put(x["state"]), dstate_out=put(x["dlast"]))
        want = ref.backward(*h, x["g"].numpy(), 1.0, lens, s, ds)
        size = ref.backward(*a, x["g"].numpy(), 1.0, lens, mag(s), mag(ds))
        for i, name in enumerate(("dq", "dk", "dv")):
            close(got[i], want[i], size[i], dtype, tokens + dk + dv + heads, name)


def test_a_state_is_read_to_more_than_bf16():
    # Nothing but the state: k and v are zeros.
    b, t, heads, dv = 6, 70, 4, 128
    gen = torch.Generator().manual_seed(61)
    q = torch.randn((b, t, heads, 1), generator=gen).bfloat16()
    state = torch.randn((b, heads, 1, dv), generator=gen)
    g = torch.from_numpy(decays(heads))
    g[heads // 2] = -0.5
    zero = torch.zeros((b, t, heads, dv), dtype=torch.bfloat16)
    out, _ = ps.linattn(q.cuda(), zero[..., :1].cuda(), zero.cuda(), g.cuda(), state=state.cuda())
    flat = lambda x: x.reshape((-1,) + x.shape[2:])  # noqa: E731
    want, _ = ref.forward(host(flat(q)), host(flat(zero[..., :1])), host(flat(zero)), g.numpy(), 1.0, (t,) * b,
                          host(state))
    close(out, want, np.abs(want), "bf16", t + dv + 1, "out")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_mean_error_is_the_outputs_own(dtype):
    # Against the definition rounded once: root mean squares.  A rounding to
    # nearest has r = rms(rounded - exact); the kernel's parts add 2^-14 A at
    # most to each, of either sign, and change the rounding where they cross
    # the middle of a step, which adds as much again.
    lens, heads, d = (512,), 2, 128
    x = make(lens, heads, heads, heads, d, d, dtype, 62, packed=False, state=False)
    out, _ = ps.linattn(*[dev(x, n, lens, False) for n in "qkv"], x["g"].cuda(), scale=0.125)
    want, _ = ref.forward(*[host(x[n]) for n in "qkv"], x["g"].numpy(), 0.125, lens)
    once = host(torch.from_numpy(want).to(DTYPES[dtype]))
    rms = lambda t: float(np.sqrt((t * t).mean()))  # noqa: E731
    # rms sizes: the terms are random, so A's share is 2^-14 of the output's
    assert rms(host(out).reshape(want.shape) - want) <= rms(once - want) + 2 * 2.0 ** -14 * rms(want)
