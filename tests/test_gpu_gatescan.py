"""The gated recurrence on the GPU against its definition in 64 bits.

Tolerances.  A rounding to a type moves a value by at most eps / 2 of it.  With
S the same recurrence over absolute values, a step rounds its product and sum
(2 steps of 2^-24), its gate and 1 - gate (4 each, from an exponential, a
division and their argument), and the tiles' products round each gate once
more: under 16 * 2^-24 of S for each token that a value has passed, and 16 for
the rest.  Outputs are rounded once (f16 to half its smallest number where
they are less than normal).
"""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import gatescan_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
FORMS = [(f, b) for f in ("decay", "log", "sigmoid") for b in (False, True)]


def host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def make(lens, width, dtype, form, seed=0, state=True):
    gen = torch.Generator().manual_seed(seed)
    n = sum(lens)
    z = torch.randn((n, width), generator=gen) * 2 + 2
    if form == "decay":
        gate = torch.sigmoid(z) * torch.where(torch.rand(z.shape, generator=gen) < 0.1, -1.0, 1.0)
        gate[torch.rand(z.shape, generator=gen) < 0.02] = 0.0
        gate[torch.rand(z.shape, generator=gen) < 0.05] = 1.0
    else:
        gate = torch.nn.functional.logsigmoid(z) if form == "log" else z * 2
    rows = lambda: torch.randn((n, width), generator=gen).to(DTYPES[dtype])  # noqa: E731
    states = lambda: torch.randn((len(lens), width), generator=gen) if state else None  # noqa: E731
    return {"gate": gate.to(DTYPES[dtype]), "x": rows(), "dout": rows(), "state": states(), "dlast": states()}


def near(got, want, size, dtype, tokens, what):
    got = host(got).reshape(want.shape)
    tol = HALF[dtype] * np.abs(want) + 16 * (tokens + 1) * 2.0 ** -24 * size + 1e-37
    if dtype == "fp16":
        tol = tol + 2.0 ** -25
    off = np.abs(got - want)
    assert np.isfinite(got).all(), what
    worst = np.unravel_index(np.argmax(off - tol), off.shape)
    assert (off <= tol).all(), "%s%s: off by %g where %g is allowed" % (what, worst, off[worst], tol[worst])


def on_gpu(t, lens, packed):
    """On the GPU, of equal sequences as [B, T, D]."""
    t = t.cuda()
    return t if packed else t.view((len(lens), -1) + t.shape[1:])


def check(lens, width, dtype, form, blend, packed=True, state=True, seed=0, there=on_gpu):
    """Forward and gradient; the outputs start as NaN."""
    s = make(lens, width, dtype, form, seed, state)
    dev = {k: None if v is None else v.cuda() if k in ("state", "dlast") else there(v, lens, packed)
           for k, v in s.items()}
    ends = torch.tensor(np.cumsum(lens), dtype=torch.int32).cuda() if packed else None
    nan = lambda t: torch.full_like(t, float("nan")).contiguous()  # noqa: E731
    states = torch.full((len(lens), width), float("nan"), device="cuda")
    out, last = nan(dev["x"]), states.clone()
    got = ps.gatescan(dev["gate"], dev["x"], form=form, blend=blend, ends=ends, state=dev["state"], out=out,
                      state_out=last)
    assert got[0] is out and got[1] is last
    a, rest = ref.gates(host(s["gate"]), form)
    x = host(s["x"])
    h, wlast = ref.forward(a, rest * x if blend else x, lens, host(s["state"]))
    mag = None if s["state"] is None else np.abs(host(s["state"]))
    size, slast = ref.forward(np.abs(a), np.abs(rest * x) if blend else np.abs(x), lens, mag)
    tokens = max(lens)
    near(out, h, size, dtype, tokens, "out")
    near(last, wlast, slast, "fp32", tokens, "state")

    given = torch.from_numpy(h).to(DTYPES[dtype])            # as a forward pass leaves it
    dgate, dx, dstate = nan(dev["x"]), nan(dev["x"]), states.clone()
    ps.gatescan_grad(dev["dout"], dev["gate"], dev["x"] if blend else None, there(given, lens, packed), form=form,
                     blend=blend, ends=ends, state=dev["state"], dstate_out=dev["dlast"], dgate=dgate, dx=dx,
                     dstate=dstate)
    dh, first = ref.backward(host(s["dout"]), a, lens, host(s["dlast"]))
    dmag = None if s["dlast"] is None else np.abs(host(s["dlast"]))
    dsize, sfirst = ref.backward(np.abs(host(s["dout"])), np.abs(a), lens, dmag)
    prev = ref.before(host(given), lens, host(s["state"]))
    slope = ref.slope(a, rest, form)
    near(dx, dh * rest if blend else dh, dsize * np.abs(rest) if blend else dsize, dtype, tokens, "dx")
    near(dgate, dh * (prev - x if blend else prev) * slope,
         dsize * (np.abs(prev) + (np.abs(x) if blend else 0)) * np.abs(slope), dtype, tokens, "dgate")
    near(dstate, first, sfirst, "fp32", tokens, "dstate")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("form,blend", FORMS)
@pytest.mark.parametrize("lens", [(1,), (2, 2, 2), (127, 127), (128,), (129, 129), (256,), (257,), (700, 700)])
def test_lengths(lens, form, blend, dtype):
    check(lens, 72, dtype, form, blend, packed=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("form,blend", FORMS)
@pytest.mark.parametrize("lens", [(5,), (0, 3), (1, 0, 0, 64, 1), (128, 128, 0), (65, 0, 130, 2, 0, 0),
                                  (0, 0, 600, 3, 0, 290)])
def test_packed(lens, form, blend, dtype):
    check(lens, 40, dtype, form, blend)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("width", [1, 3, 7, 8, 31, 63, 64, 65, 130, 333])
def test_widths(width, dtype):
    check((140, 31, 1), width, dtype, "sigmoid", True)
    check((150, 150), width, dtype, "log", False, packed=False, state=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_without_states(dtype):
    check((300, 0, 20), 24, dtype, "decay", False, state=False)
    check((300, 0, 20), 24, dtype, "log", True, state=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_short_sequences(dtype):
    gen = np.random.default_rng(5)
    lens = gen.integers(0, 4, 900).tolist() + [0] * 300 + [2]
    check(lens, 24, dtype, "sigmoid", True)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_long_sequences(dtype):
    # more tiles than one look back reaches, and a start in the middle of some
    check((9001,), 3, dtype, "sigmoid", False, packed=False)
    check((3000, 5003, 1, 4000), 5, dtype, "log", True)


def strided(t, lens, packed):
    """Rows two apart of a wider tensor, that start off every alignment but the element's."""
    t = on_gpu(t, lens, packed)
    wide = torch.full(t.shape[:-2] + (2 * t.shape[-2], t.shape[-1] + 5), float("nan"), dtype=t.dtype, device="cuda")
    view = wide[..., ::2, 3:3 + t.shape[-1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("width", [9, 64])
def test_strides(width, dtype):
    check((140, 140), width, dtype, "sigmoid", True, packed=False, there=strided)
    check((140, 0, 33), width, dtype, "log", True, there=strided)


def test_a_broadcast_gate():
    # one gate for all sequences, by a stride of zero, and sequences turned about
    gate = torch.rand(1, 200, 48, device="cuda").expand(3, -1, -1)
    x = torch.randn(200, 3, 48, device="cuda").transpose(0, 1)
    got, _ = ps.gatescan(gate, x)
    want, _ = ps.gatescan(gate.contiguous(), x.contiguous())
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_no_tokens(dtype):
    state = torch.randn(3, 33, device="cuda")
    for ends in (None, torch.zeros(3, dtype=torch.int32, device="cuda")):
        rows = torch.zeros((3, 0, 33) if ends is None else (0, 33), dtype=DTYPES[dtype], device="cuda")
        out, last = ps.gatescan(rows, rows, ends=ends, state=state, want_state=True)
        assert out.shape == rows.shape and torch.equal(last, state)
        assert not ps.gatescan(rows, rows, ends=ends, want_state=True)[1].any()
        _, _, first = ps.gatescan_grad(rows, rows, None, rows, ends=ends, dstate_out=state, want_dstate=True)
        assert torch.equal(first, state)
    none = torch.zeros(0, 5, 8, device="cuda")
    assert ps.gatescan(none, none, want_state=True)[1].shape == (0, 8)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("used", [0, 1, 100, 128, 301])
def test_rows_past_the_last_end(used, dtype):
    # What is in no sequence is not read; given outputs stay as they are there, new ones are zeros.
    n, d = 900, 40
    s = make((n,), d, dtype, "sigmoid")
    gate, x, dout = (s[k].cuda() for k in ("gate", "x", "dout"))
    ends = torch.tensor([used // 2, used], dtype=torch.int32, device="cuda")
    clean = [t[:used].contiguous() for t in (gate, x, dout)]
    for t in (gate, x, dout):
        t[used:] = float("nan")
    kept = torch.full_like(x, 7.0)
    out, last = ps.gatescan(gate, x, "sigmoid", True, ends=ends, out=kept, want_state=True)
    assert bool((kept[used:] == 7).all())
    fresh, _ = ps.gatescan(gate, x, "sigmoid", True, ends=ends)
    assert torch.equal(fresh[:used], out[:used]) and not fresh[used:].any()
    assert bool(torch.isfinite(last).all())
    if used:
        want, wlast = ps.gatescan(clean[0], clean[1], "sigmoid", True, ends=ends, want_state=True)
        assert torch.equal(out[:used], want) and torch.equal(last, wlast)
    given = [torch.full_like(x, 7.0) for _ in range(2)]
    h = out.clone()
    h[used:] = float("nan")
    ps.gatescan_grad(dout, gate, x, h, "sigmoid", True, ends=ends, dgate=given[0], dx=given[1])
    new = ps.gatescan_grad(dout, gate, x, h, "sigmoid", True, ends=ends)
    half = ps.gatescan_grad(dout, gate, x, h, "sigmoid", True, ends=ends, dx=given[1])
    for g, f, m in zip(given, new, half):
        assert bool((g[used:] == 7).all()) and torch.equal(g[:used], f[:used]) and torch.equal(m[:used], f[:used])
        assert not f[used:].any() and bool(torch.isfinite(f).all())
    assert not half[0][used:].any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_is_not_finite_stays_where_it_is(bad, dtype):
    # an infinity decays to itself, over many tiles; no other channel, sequence or earlier token sees it
    n, d = 2000, 20
    gate = torch.full((n, d), 0.25, dtype=DTYPES[dtype], device="cuda")
    x = torch.ones_like(gate)
    x[700, 7] = bad
    ends = torch.tensor([650, 1900, 2000], dtype=torch.int32, device="cuda")
    out, last = ps.gatescan(gate, x, ends=ends, want_state=True)
    inside = torch.zeros_like(out, dtype=torch.bool)
    inside[700:1900, 7] = True
    same = torch.isinf if bad > 0 else torch.isnan
    assert bool(same(out[inside]).all()) and bool(torch.isfinite(out[~inside]).all())
    assert bool(same(last[1, 7])) and int((~torch.isfinite(last)).sum()) == 1
    dout = torch.ones_like(gate)
    dout[1500, 3] = bad
    fine, _ = ps.gatescan(gate, torch.ones_like(gate), ends=ends)
    dgate, dx, dstate = ps.gatescan_grad(dout, gate, None, fine, ends=ends, want_dstate=True)
    inside.zero_()
    inside[650:1501, 3] = True
    assert bool(same(dx[inside]).all()) and bool(torch.isfinite(dx[~inside]).all())
    assert bool(torch.isfinite(dgate[~inside]).all())
    assert bool(same(dstate[1, 3])) and int((~torch.isfinite(dstate)).sum()) == 1


@pytest.mark.parametrize("form", ["log", "sigmoid"])
def test_gates_at_their_ends(form):
    # a of 0 and 1, exactly, and no tokens lost between
    d = 8
    gate = torch.tensor([float("-inf"), -1e30, -300.0, -90.0, 0.0, -0.0])
    if form == "sigmoid":
        gate = torch.cat([gate[:4], torch.tensor([300.0, float("inf")])])
    gate = gate.view(-1, 1).repeat(1, d).cuda()
    x = torch.full_like(gate, 2.0)
    state = torch.full((1, d), 3.0, device="cuda")
    for blend in (False, True):
        out, _ = ps.gatescan(gate[None], x[None], form, blend, state=state)
        assert out[0, :, 0].tolist() == ([2.0] * 6 if blend else [2.0] * 4 + [4.0, 6.0])
    # a gate close to 1 keeps what it should of long memories: 1 - a is good to its last bits
    g = torch.full((1, 4000, d), 12.0 if form == "sigmoid" else -6e-6, device="cuda")
    out, _ = ps.gatescan(g, torch.ones_like(g), form, True)
    a, rest = ref.gates(host(g)[0], form)
    want, _ = ref.forward(a, rest, [4000])
    assert np.abs(host(out)[0] - want).max() <= 4000 * 2.0 ** -24 * want.max()


def test_the_same_bits_every_time():
    s = make((40000,), 192, "bf16", "sigmoid")
    gate, x = s["gate"].cuda()[None], s["x"].cuda()[None]
    out, last = ps.gatescan(gate, x, "sigmoid", True, want_state=True)
    grads = ps.gatescan_grad(x, gate, x, out, "sigmoid", True)
    for _ in range(8):
        again = ps.gatescan(gate, x, "sigmoid", True, want_state=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], last)
        for g, w in zip(ps.gatescan_grad(x, gate, x, out, "sigmoid", True)[:2], grads):
            assert torch.equal(g, w)


def test_ends_that_fall_stay_in_bounds():
    # no batch: unspecified values, but nothing outside the rows is touched and the call ends
    buf = torch.full((3, 700, 24), 5.0, device="cuda")
    rows = torch.rand(700, 24, device="cuda")
    for ends in ([500, 100, 700], [0, 900, 3], [700, 0], [5, 4, 3, 2, 1, 0], [300, 2 ** 31 - 1, 10]):
        e = torch.tensor(ends, dtype=torch.int32, device="cuda")
        out, states = buf[1], torch.full((len(ends) + 2, 24), 5.0, device="cuda")
        ps.gatescan(rows, rows, ends=e, out=out, state_out=states[1:-1])
        ps.gatescan_grad(rows, rows, None, rows, ends=e, dgate=out, dx=torch.empty_like(rows),
                         dstate=states[1:-1])
        torch.cuda.synchronize()
        assert bool((buf[0] == 5).all()) and bool((buf[2] == 5).all())
        assert bool((states[0] == 5).all()) and bool((states[-1] == 5).all())


# --------------------------------------------------------------------------
# Single tokens
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("form,blend", FORMS)
@pytest.mark.parametrize("rows,width,pool", [(1, 64, 0), (3, 7, 0), (5, 33, 9), (40, 1000, 50), (17, 264, 17)])
def test_steps(rows, width, pool, form, blend, dtype):
    s = make((1,) * rows, width, dtype, form)
    gen = torch.Generator().manual_seed(8)
    state = torch.randn((pool or rows, width), generator=gen)
    slots = torch.randperm(pool, generator=gen)[:rows].to(torch.int32) if pool else None
    if pool:
        slots[rows // 2], slots[rows - 1] = -1, pool
    a, rest = ref.gates(host(s["gate"]), form)
    b = rest * host(s["x"]) if blend else host(s["x"])
    want, wout = host(state), np.zeros((rows, width))
    size, sout = np.abs(want), np.zeros((rows, width))
    for r in range(rows):
        at = r if slots is None else int(slots[r])
        if 0 <= at < len(want):
            want[at] = wout[r] = a[r] * want[at] + b[r]
            size[at] = sout[r] = np.abs(a[r]) * size[at] + np.abs(b[r])
    for apart in (False, True):
        pool_in = state.cuda()
        pool_out = torch.full_like(pool_in, 9.0) if apart else None
        out, got = ps.gatescan_step(s["gate"].cuda(), s["x"].cuda(), pool_in, form, blend,
                                    None if slots is None else slots.cuda(), state_out=pool_out)
        assert got is (pool_out if apart else pool_in)
        near(out, wout, sout, dtype, 1, "out")
        used = np.ones(len(want), dtype=bool) if slots is None else np.isin(np.arange(len(want)), slots.numpy())
        near(got[torch.from_numpy(used).cuda()], want[used], size[used], "fp32", 1, "state")
        rest_of = host(got)[~used]
        assert np.array_equal(rest_of, np.full_like(rest_of, 9.0) if apart else host(state)[~used])
        if apart:
            assert torch.equal(pool_in.cpu(), state)


def test_steps_follow_a_sequence():
    # the states that gatescan leaves go on as tokens one at a time
    s = make((50, 50), 96, "bf16", "sigmoid")
    gate, x = (s[k].cuda().view(2, 50, 96) for k in ("gate", "x"))
    whole, last = ps.gatescan(gate, x, "sigmoid", True, want_state=True)
    part, state = ps.gatescan(gate[:, :30], x[:, :30], "sigmoid", True, want_state=True)
    for t in range(30, 50):
        out, _ = ps.gatescan_step(gate[:, t], x[:, t], state, "sigmoid", True)
        near(out, host(whole[:, t]), np.abs(host(whole[:, t])) + 1, "bf16", 50, "step %d" % t)
    near(state, host(last), np.abs(host(last)) + 1, "fp32", 50, "state")


# --------------------------------------------------------------------------
# Streams and graphs
# --------------------------------------------------------------------------

def test_captured_and_replayed_beside_eager_calls():
    s = make((3000,), 130, "bf16", "log")
    gate, x, dout = (s[k].cuda()[None] for k in ("gate", "x", "dout"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, last = ps.gatescan(gate, x, "log", True, want_state=True)
        grads = ps.gatescan_grad(dout, gate, x, out, "log", True)[:2]
        want = [t.clone() for t in (out, last, *grads)]
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out, last = ps.gatescan(gate, x, "log", True, want_state=True)
            grads = ps.gatescan_grad(dout, gate, x, out, "log", True)[:2]
        for i in range(4):
            for t in (out, last, *grads):
                t.fill_(float("nan"))
            # the same buffer, in other layouts, between the replays
            ps.radix_perm_u32(torch.arange(50000, dtype=torch.int32, device="cuda"))
            ps.gatescan(gate[:, :1000 + i], x[:, :1000 + i], "log")
            graph.replay()
            side.synchronize()
            for t, w in zip((out, last, *grads), want):
                assert torch.equal(t, w)


def test_on_another_stream():
    s = make((500, 500), 64, "bf16", "sigmoid")
    gate, x = (s[k].cuda().view(2, 500, 64) for k in ("gate", "x"))
    want, _ = ps.gatescan(gate, x, "sigmoid")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = ps.gatescan(gate, x, "sigmoid", stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_gradients_are_refused_and_autograd_goes_through():
    gate = torch.rand(2, 40, 16, device="cuda", requires_grad=True)
    x = torch.randn(2, 40, 16, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="gradient"):
        ps.gatescan(gate, x)

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, gate, x):
            out = ps.gatescan(gate, x, "sigmoid", True)[0]
            ctx.save_for_backward(gate, x, out)
            return out

        @staticmethod
        def backward(ctx, dout):
            return ps.gatescan_grad(dout.contiguous(), *ctx.saved_tensors, form="sigmoid", blend=True)[:2]

    Scan.apply(gate, x).square().sum().backward()
    a = torch.sigmoid(gate.detach().double()).requires_grad_()
    y = x.detach().double().requires_grad_()
    h, total = torch.zeros(2, 16, dtype=torch.float64, device="cuda"), 0
    for t in range(40):
        h = a[:, t] * h + (1 - a[:, t]) * y[:, t]
        total = total + h.square().sum()
    total.backward()
    slope = (a * (1 - a)).detach()
    assert torch.allclose(gate.grad.double(), a.grad * slope, rtol=1e-5, atol=1e-6)
    assert torch.allclose(x.grad.double(), y.grad, rtol=1e-5, atol=1e-6)
