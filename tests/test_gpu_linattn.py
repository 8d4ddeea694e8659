"""Linear attention with decay on the GPU against its definition in 64 bits.

Tolerances.  A rounding to a type moves a value by at most h = eps / 2 of it.
With A the same sums taken over absolute values, an output may be off by
    h |out|                      its own rounding,
    2 H A                        scores and state rounded to bf16 before they
                                 are multiplied (H = 2^-8; bf16 rows only),
    (tokens + widths + 128) 2^-23 A    the 32-bit sums and powers.
States and their gradients are never rounded below 32 bits.  Where heads
share an input, A is summed over them too.
"""
import ctypes

import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
SCALE = 0.125


def decays(heads):
    """No decay, no memory, and all between."""
    g = np.log1p(-2.0 ** -np.linspace(1.0, 11.0, heads))
    g[0] = 0.0
    if heads > 2:
        g[heads // 2] = -np.inf
    return g.astype(np.float32)


def make(lens, heads, hk, hv, dk, dv, dtype, seed=0, packed=True, state=True):
    gen = torch.Generator().manual_seed(seed)
    n = sum(lens)
    mk = lambda *s: torch.randn(s, generator=gen).to(DTYPES[dtype])  # noqa: E731
    x = {"q": mk(n, heads, dk), "k": mk(n, hk, dk), "v": mk(n, hv, dv), "do": mk(n, heads, dv)}
    x["g"] = torch.from_numpy(decays(heads))
    x["state"] = torch.randn((len(lens), heads, dk, dv), generator=gen) if state else None
    x["dlast"] = torch.randn((len(lens), heads, dk, dv), generator=gen) if state else None
    x["ends"] = torch.tensor(np.cumsum(lens), dtype=torch.int32) if packed else None
    return x


def host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def dev(x, name, lens, packed):
    t = x[name].cuda()
    return t if packed else t.view((len(lens), -1) + t.shape[1:])


def near(got, want, size, dtype, terms, what, state=False):
    """`got` within the tolerance of `want`; `size`: the sums over absolute values."""
    got = host(got).reshape(want.shape)
    h = HALF["fp32" if state else dtype]
    inner = 2.0 * HALF["bf16"] if dtype == "bf16" and not state else 0.0
    tol = h * np.abs(want) + (inner + (terms + 128) * 2.0 ** -23) * size + 1e-30
    if dtype == "fp16" and not state:
        tol = tol + 2.0 ** -25               # half a step of fp16's subnormal numbers
    off = np.abs(got - want)
    assert np.isfinite(got).all(), what
    assert (off <= tol).all(), "%s: off by %g where %g is allowed" % (
        what, off.flat[np.argmax(off - tol)], tol.flat[np.argmax(off - tol)])


def check_forward(lens, heads, hk, hv, dk, dv, dtype, packed=True, state=True, seed=0):
    x = make(lens, heads, hk, hv, dk, dv, dtype, seed, packed, state)
    args = [dev(x, n, lens, packed) for n in "qkv"]
    out = torch.full(args[0].shape[:-1] + (dv,), float("nan"), dtype=args[0].dtype, device="cuda")
    last = torch.full((len(lens), heads, dk, dv), float("nan"), device="cuda")
    ps.linattn(*args, x["g"].cuda(), scale=SCALE, ends=x["ends"].cuda() if packed else None,
               state=x["state"].cuda() if state else None, out=out, state_out=last)
    want, wlast = ref.forward(host(x["q"]), host(x["k"]), host(x["v"]), x["g"].numpy(), SCALE, lens,
                              host(x["state"]))
    a = [np.abs(host(x[n])) for n in "qkv"]
    size, slast = ref.forward(*a, x["g"].numpy(), SCALE, lens,
                              np.abs(host(x["state"])) if state else None)
    terms = max(lens) + dk + dv
    near(out, want, size, dtype, terms, "out")
    near(last, wlast, slast, dtype, terms, "state", state=True)


def check_backward(lens, heads, hk, hv, dk, dv, dtype, packed=True, state=True, seed=0):
    x = make(lens, heads, hk, hv, dk, dv, dtype, seed, packed, state)
    args = [dev(x, n, lens, packed) for n in ("do", "q", "k", "v")]
    nan = lambda t: torch.full_like(t, float("nan"))  # noqa: E731
    outs = [nan(t) for t in args[1:]]
    ds = torch.full((len(lens), heads, dk, dv), float("nan"), device="cuda")
    ps.linattn_grad(*args, x["g"].cuda(), scale=SCALE, ends=x["ends"].cuda() if packed else None,
                    state=x["state"].cuda() if state else None,
                    dstate_out=x["dlast"].cuda() if state else None,
                    dq=outs[0], dk=outs[1], dv=outs[2], dstate=ds)
    names = ("do", "q", "k", "v")
    want = ref.backward(*[host(x[n]) for n in names], x["g"].numpy(), SCALE, lens,
                        host(x["state"]), host(x["dlast"]))
    size = ref.backward(*[np.abs(host(x[n])) for n in names], x["g"].numpy(), SCALE, lens,
                        np.abs(host(x["state"])) if state else None,
                        np.abs(host(x["dlast"])) if state else None)
    terms = max(lens) + dk + dv + heads
    for got, w, s, name in zip(outs, want, size, ("dq", "dk", "dv")):
        near(got, w, s, dtype, terms, name)
    near(ds, want[3], size[3], dtype, terms, "dstate", state=True)


LENGTHS = [(1,), (2, 2), (31, 31), (32,), (33,), (64,), (65,), (130, 130), (300,), (700,)]
RAGGED = [(5,), (0, 3), (1, 0, 0, 64, 1), (65, 0, 130, 2), (600, 3, 0, 290), (0, 0)]
SHAPES = [(2, 2, 2, 64, 64), (3, 3, 3, 128, 128), (4, 2, 1, 32, 96), (6, 3, 6, 72, 40),
          (2, 1, 2, 1, 1), (3, 1, 3, 17, 63), (2, 2, 2, 128, 8), (2, 2, 2, 65, 127)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", LENGTHS)
def test_forward_lengths(lens, dtype):
    check_forward(lens, 3, 3, 3, 64, 64, dtype, packed=False)
    check_forward(lens, 2, 1, 2, 128, 72, dtype, packed=False, state=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", RAGGED)
def test_forward_packed(lens, dtype):
    check_forward(lens, 3, 3, 3, 64, 64, dtype)
    check_forward(lens, 2, 2, 1, 96, 128, dtype, state=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_widths_and_shared_heads(shape, dtype):
    check_forward((70, 0, 41), *shape, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", LENGTHS)
def test_gradient_lengths(lens, dtype):
    check_backward(lens, 3, 3, 3, 64, 64, dtype, packed=False)
    check_backward(lens, 2, 2, 2, 128, 72, dtype, packed=False, state=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", RAGGED)
def test_gradient_packed(lens, dtype):
    check_backward(lens, 3, 3, 3, 64, 64, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_gradient_widths_and_shared_heads(shape, dtype):
    check_backward((70, 0, 41), *shape, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_many_heads_cut_into_segments(dtype):
    # 96 heads of 900 and 1500 tokens: more tokens than one workgroup takes.
    check_forward((1500, 7, 900), 24, 24, 24, 64, 64, dtype)
    check_backward((1100, 7, 600), 24, 24, 24, 32, 64, dtype)


def test_gradient_is_the_difference_of_the_forward_pass():
    # The outputs are linear in each input: a step of any size is exact, up
    # to the 32-bit sums of both sides.
    lens, heads = (150, 40), 4
    x = make(lens, heads, 2, 4, 48, 32, "fp32", 3)
    put = {n: x[n].cuda() for n in ("q", "k", "v", "state", "g", "ends", "do", "dlast")}

    def loss(y):
        out, last = ps.linattn(y["q"], y["k"], y["v"], y["g"], scale=SCALE, ends=y["ends"],
                               state=y["state"], want_state=True)
        return float((out.double() * y["do"]).sum() + (last.double() * y["dlast"]).sum())

    grads = ps.linattn_grad(put["do"], put["q"], put["k"], put["v"], put["g"], scale=SCALE,
                            ends=put["ends"], state=put["state"], dstate_out=put["dlast"],
                            want_dstate=True)
    at = loss(put)
    for name, grad in zip(("q", "k", "v", "state"), grads):
        d = torch.randn(put[name].shape, generator=torch.Generator().manual_seed(9)).cuda()
        moved = dict(put)
        moved[name] = put[name] + d
        want = float((grad.double() * d).sum())
        # each loss is a sum of n products good to (tokens + widths + 128) 2^-23 of their sizes;
        # sizes here are below 2^10 and their errors random, so 2^-23 * 400 * 2^10 * sqrt(n)
        n = put["do"].numel() + put["dlast"].numel()
        assert abs(loss(moved) - at - want) <= 400 * 2.0 ** -13 * n ** 0.5, name


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strides_and_odd_offsets(dtype):
    # q, k and v as slices of one projection, tokens the inner axis of
    # another, and rows that start on no 16-byte boundary.
    b, t, h, d = 2, 75, 3, 40
    gen = torch.Generator().manual_seed(5)
    qkv = torch.randn((b, t, 3 * h * d + 1), generator=gen).to(DTYPES[dtype]).cuda()
    views = [qkv[:, :, 1 + i * h * d:1 + (i + 1) * h * d].unflatten(2, (h, d)) for i in range(3)]
    swapped = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in views]
    g = torch.from_numpy(decays(h)).cuda()
    plain = [x.contiguous() for x in views]
    want, last = ps.linattn(*plain, g, scale=SCALE, want_state=True)
    grads = ps.linattn_grad(plain[2], *plain, g, scale=SCALE)
    for xs in (views, swapped):
        out = torch.full((b, h, t, d), 7.0, dtype=qkv.dtype, device="cuda").transpose(1, 2)
        got, state = ps.linattn(*xs, g, scale=SCALE, out=out, want_state=True)
        assert torch.equal(got, want) and torch.equal(state, last)
        for a, b_ in zip(ps.linattn_grad(xs[2], *xs, g, scale=SCALE)[:3], grads[:3]):
            assert torch.equal(a, b_)
    one = plain[0][:, :, :1].expand(b, t, h, d)          # one head broadcast by a stride of 0
    a, _ = ps.linattn(one, *plain[1:], g, scale=SCALE)
    c, _ = ps.linattn(one.contiguous(), *plain[1:], g, scale=SCALE)
    assert torch.equal(a, c)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_values_that_are_not_finite_reach_no_earlier_token(bad, dtype):
    lens = (100, 90)
    x = make(lens, 2, 2, 2, 64, 64, dtype, 4)
    g = torch.tensor([-0.01, 0.0]).cuda()
    y = {n: x[n].cuda() for n in ("q", "k", "v", "state", "ends")}
    clean, _ = ps.linattn(y["q"], y["k"], y["v"], g, scale=SCALE, ends=y["ends"], state=y["state"])
    for name in ("q", "k", "v"):
        z = dict(y)
        z[name] = y[name].clone()
        z[name][57, 1, 5] = bad
        out, last = ps.linattn(z["q"], z["k"], z["v"], g, scale=SCALE, ends=y["ends"],
                               state=y["state"], want_state=True)
        mask = torch.ones_like(out, dtype=torch.bool)
        mask[57:(58 if name == "q" else 100), 1] = False
        h = HALF[dtype] if dtype != "fp32" else 0.0
        # a chunk taken token by token adds its terms in another order
        size = float(clean.float().abs().max())
        assert torch.isfinite(out[mask]).all(), name
        off = (out[mask].float() - clean[mask].float()).abs().max()
        assert off <= (6 * h + 2.0 ** -16) * size, name
        assert not torch.isfinite(out[57, 1]).all(), name
        assert torch.isfinite(last[1]).all() and torch.isfinite(last[0, 0]).all()
        assert torch.isfinite(last[0, 1]).all() == (name == "q"), name


def test_rows_outside_every_sequence_are_left_alone():
    x = make((40, 30), 2, 2, 2, 64, 64, "bf16", 6)
    g = x["g"].cuda()
    q, k, v = (x[n].cuda() for n in "qkv")
    for t in (q, k, v):
        t[60:] = float("nan")
    ends = torch.tensor([40, 60], dtype=torch.int32).cuda()
    out = torch.full_like(v, 9.0)
    ps.linattn(q, k, v, g, ends=ends, out=out)
    assert torch.isfinite(out).all() and (out[60:] == 9).all()
    # ends that fall, and ends past the rows, are cut to the rows
    for e in ((40, 20), (40, 1 << 30), (-1, 3)):
        ps.linattn(q, k, v, g, ends=torch.tensor(e, dtype=torch.int32).cuda(), out=out, want_state=True)
    torch.cuda.synchronize()


def test_nothing_to_do():
    g = torch.zeros(2, device="cuda")
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    out, last = ps.linattn(e(0, 5, 2, 8), e(0, 5, 2, 8), e(0, 5, 2, 8), g, want_state=True)
    assert out.shape == (0, 5, 2, 8) and last.shape == (0, 2, 8, 8)
    s = torch.randn(3, 2, 8, 8, device="cuda")
    out, last = ps.linattn(e(3, 0, 2, 8), e(3, 0, 2, 8), e(3, 0, 2, 8), g, state=s, want_state=True)
    assert torch.equal(last, s)
    d = ps.linattn_grad(e(3, 0, 2, 8), e(3, 0, 2, 8), e(3, 0, 2, 8), e(3, 0, 2, 8), g,
                        dstate_out=s, want_dstate=True)
    assert torch.equal(d[3], s)
    out, _ = ps.linattn_step(e(0, 2, 8), e(0, 2, 8), e(0, 2, 8), g, e(0, 2, 8, 8))
    assert out.shape == (0, 2, 8)


# --------------------------------------------------------------------------
# Single tokens
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES + [(16, 16, 16, 128, 128)])
@pytest.mark.parametrize("rows", [1, 3, 70])
def test_step_matches_the_definition(rows, shape, dtype):
    heads, hk, hv, dk, dv = shape
    x = make((1,) * rows, heads, hk, hv, dk, dv, dtype, 7)
    pool = rows + 5
    gen = torch.Generator().manual_seed(8)
    states = torch.randn((pool, heads, dk, dv), generator=gen)
    slots = torch.randperm(pool, generator=gen)[:rows].int()
    idle = list(range(1, rows, 4))
    slots[idle] = torch.tensor([-1, pool, -2 ** 31, 2 ** 31 - 1] * rows)[:len(idle)].int()
    args = [x[n].cuda() for n in "qkv"] + [x["g"].cuda()]
    live = [r for r in range(rows) if r not in idle]
    pick = states[slots[live].long()]
    sel = {n: host(x[n][live]) for n in "qkv"}
    want, new = ref.forward(sel["q"], sel["k"], sel["v"], x["g"].numpy(), SCALE, (1,) * len(live), host(pick))
    size, snew = ref.forward(*[np.abs(sel[n]) for n in "qkv"], x["g"].numpy(), SCALE,
                             (1,) * len(live), np.abs(host(pick)))
    into = torch.full_like(states, float("nan")).cuda()
    out = torch.full((rows, heads, dv), float("nan"), dtype=DTYPES[dtype]).cuda()
    ps.linattn_step(*args, states.cuda(), scale=SCALE, slots=slots.cuda(), out=out, state_out=into)
    here = states.cuda()
    out2, same = ps.linattn_step(*args, here, scale=SCALE, slots=slots.cuda())
    assert same is here and torch.equal(out, out2)
    touched = slots[live].long()
    near(out[live], want, size, "fp32" if dtype == "fp32" else "fp16" if dtype == "fp16" else "bf16",
         dk, "out")
    near(into[touched.cuda()], new, snew, dtype, 1, "state", state=True)
    assert torch.equal(here[touched.cuda()], into[touched.cuda()])
    rest = [i for i in range(pool) if i not in touched.tolist()]
    assert torch.isnan(into[rest]).all() and torch.equal(here[rest].cpu(), states[rest])
    assert (out[idle] == 0).all()


def test_steps_follow_the_prompt():
    # A prompt, then tokens one by one, against the whole sequence at once.
    x = make((90, 90), 3, 3, 3, 64, 64, "fp32", 10, packed=False, state=False)
    q, k, v = (dev(x, n, (90, 90), False) for n in "qkv")
    g = x["g"].cuda()
    whole, last = ps.linattn(q, k, v, g, scale=SCALE, want_state=True)
    _, state = ps.linattn(q[:, :80], k[:, :80], v[:, :80], g, scale=SCALE, want_state=True)
    for t in range(80, 90):
        out, state = ps.linattn_step(q[:, t], k[:, t], v[:, t], g, state, scale=SCALE)
        assert torch.allclose(out, whole[:, t], rtol=2.0 ** -13, atol=2.0 ** -10)
    assert torch.allclose(state, last, rtol=2.0 ** -13, atol=2.0 ** -10)


def test_step_takes_any_strides():
    rows, heads, d = 6, 4, 32
    qkv = torch.randn(rows, 3 * heads * d + 3, device="cuda")
    views = [qkv[:, i * heads * d + i:(i + 1) * heads * d + i].unflatten(1, (heads, d)) for i in range(3)]
    g = torch.from_numpy(decays(heads)).cuda()
    s = torch.randn(rows, heads, d, d, device="cuda")
    a, sa = ps.linattn_step(*[x.contiguous() for x in views], g, s.clone())
    out = torch.empty(heads, rows, d, device="cuda").transpose(0, 1)
    b, sb = ps.linattn_step(*views, g, s.clone(), out=out)
    assert torch.equal(a, b) and torch.equal(sa, sb)
    flat = torch.empty(s.numel() + 1, device="cuda")       # a state that starts on 4 bytes only
    odd = flat[1:].view_as(s).copy_(s)
    c, sc = ps.linattn_step(*views, g, odd)
    assert torch.allclose(a, c, rtol=1e-5, atol=1e-4) and torch.allclose(sa, sc)


# --------------------------------------------------------------------------
# Streams and graphs
# --------------------------------------------------------------------------

def test_another_stream():
    x = make((300, 200), 4, 4, 4, 64, 64, "bf16", 11)
    args = [x[n].cuda() for n in "qkv"] + [x["g"].cuda()]
    kw = dict(scale=SCALE, ends=x["ends"].cuda(), state=x["state"].cuda(), want_state=True)
    want = ps.linattn(*args, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ps.linattn(*args, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed():
    lens = (700, 3, 500)
    x = make(lens, 8, 8, 2, 64, 64, "bf16", 12)
    y = {n: x[n].cuda() for n in ("do", "q", "k", "v", "state", "dlast", "ends", "g")}
    outs = {n: torch.empty_like(y["do" if n == "out" else n[1:]]) for n in ("out", "dq", "dk", "dv")}
    last, ds = torch.empty_like(y["state"]), torch.empty_like(y["state"])
    pool = y["state"].clone()
    step = torch.empty_like(y["do"][:3])

    def calls():
        ps.linattn(y["q"], y["k"], y["v"], y["g"], scale=SCALE, ends=y["ends"], state=y["state"],
                   out=outs["out"], state_out=last)
        ps.linattn_grad(y["do"], y["q"], y["k"], y["v"], y["g"], scale=SCALE, ends=y["ends"],
                        state=y["state"], dstate_out=y["dlast"], dq=outs["dq"], dk=outs["dk"],
                        dv=outs["dv"], dstate=ds)
        ps.linattn_step(y["q"][:3], y["k"][:3], y["v"][:3], y["g"], pool, scale=SCALE, out=step)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    results = list(outs.values()) + [last, ds, pool, step]
    for rep in range(4):
        for n in ("q", "k", "v", "do"):
            y[n].copy_(torch.randn(y[n].shape, generator=torch.Generator().manual_seed(rep)))
        pool.copy_(y["state"])
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            calls()
        torch.cuda.synchronize()
        want = [t.clone() for t in results]
        for t in results:
            t.fill_(float("nan"))
        pool.copy_(y["state"])
        # other eager work of the library on the same scratch buffer
        with torch.cuda.stream(stream):
            ps.scan_exclusive_u32(torch.arange(100000, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(results, want):
            assert torch.equal(a, b), rep


# --------------------------------------------------------------------------
# Positions past 32 bits
# --------------------------------------------------------------------------

def test_offsets_past_32_bits():
    # Token rows 2^25 elements apart: the last of 100 tokens starts past 2^31
    # elements, and past 2^32 bytes.
    t, step = 100, 1 << 25
    buf = torch.empty(t * step, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((1, t, 2, 32), (0, step, 32, 1))
    near_ = torch.randn(1, t, 2, 32, device="cuda").bfloat16()
    far.copy_(near_)
    g = torch.tensor([-0.1, -0.01], device="cuda")
    want, _ = ps.linattn(near_, near_, near_, g)
    got, _ = ps.linattn(far, far, far, g, out=buf.as_strided((1, t, 2, 32), (0, step, 32, 1), 64))
    assert torch.equal(got, want)
    for a, b in zip(ps.linattn_grad(far, far, far, far, g)[:3],
                    ps.linattn_grad(near_, near_, near_, near_, g)[:3]):
        assert torch.equal(a, b)


# --------------------------------------------------------------------------
# Refusals of the binding
# --------------------------------------------------------------------------

def test_bad_tensors_are_refused():
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    q, g, s = z(2, 5, 4, 8), z(4), z(2, 4, 8, 8)
    for args in ((z(2, 5, 4, 8).half(), q, q, g), (q, q, q.bfloat16(), g), (q, q, q, g.double()),
                 (q, q, q, None)):
        with pytest.raises(TypeError):
            ps.linattn(*args)
    for args in ((q, z(2, 5, 3, 8), q, g), (q, z(2, 5, 4, 9), q, g), (q, z(2, 6, 4, 8), q, g),
                 (q[0], q[0], q[0], g), (z(2, 5, 4, 129), z(2, 5, 4, 129), q, g),
                 (q.transpose(2, 3), q, q, g), (q, q, q, g.cpu()), (q, q, q, z(2))):
        with pytest.raises(ValueError):
            ps.linattn(*args)
    for kw in (dict(state=z(2, 4, 8, 7)), dict(state=z(3, 4, 8, 8)), dict(out=z(2, 5, 4, 9)),
               dict(state_out=s.transpose(2, 3)), dict(state=s.cpu())):
        with pytest.raises(ValueError):
            ps.linattn(q, q, q, g, **kw)
    with pytest.raises(ps.LibscanError):
        ps.linattn(q, q, q, g, state=s, state_out=s)
    with pytest.raises(TypeError):
        ps.linattn(q, q, q, g, state=s.half())
    with pytest.raises(ValueError):
        ps.linattn_grad(z(2, 5, 4, 9), q, q, q, g)
    p = z(2, 4, 8)
    for kw in (dict(state=z(3, 4, 8, 8)), dict(state=s, slots=z(3, dtype=torch.int32)),
               dict(state=s, state_out=z(3, 4, 8, 8)), dict(state=s, out=z(2, 4, 7))):
        with pytest.raises(ValueError):
            ps.linattn_step(p, p, p, g, **kw)
    with pytest.raises(TypeError):
        ps.linattn_step(p, p, p, g, s, slots=z(2, dtype=torch.int64))
    x, u = z(3, 50), z(3)
    for args, kw in (((x, z(4)), {}), ((x, u.cpu()), {}), ((x, u), dict(top_p=z(2))),
                     ((x[0], u), {}), ((x.t(), z(50)), {}), ((x, u), dict(tokens=z(2, dtype=torch.int32)))):
        with pytest.raises(ValueError):
            ps.sample_logits(*args, **kw)
    for kw in (dict(top_k=z(3)), dict(temperature=z(3).half()), dict(kept=z(3))):
        with pytest.raises(TypeError):
            ps.sample_logits(x, u, **kw)
