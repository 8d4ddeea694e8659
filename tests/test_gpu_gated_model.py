"""Embedding rows, gated recurrences, penalties and sampling together, as a
recurrent model trains and serves, beside other calls on their streams'
scratch, and long lists of penalties.

Tolerances.  u = 2^-24 is half a step of 32 bits, K the width of the products,
T the tokens of a sequence.  With S the same computation over absolute values:
a gate's argument is off by K u of its sum of absolute values, at most G, and
its sigmoid moves by a quarter of that at most, 1 - gate relative to itself by
all of it, so that a gate and its rest are off by (K G + 8) u of themselves.
A recurrence's value or gradient has passed T gates at most, each with a product
and a sum more; two of them, the products' K + 1 steps on either side and
T additions of rows of one id make T (K G + 10) + T (K G + 10) + 2 (K + 1) + T
steps, counted twice for what is of higher order.
"""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import gatescan_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids):
        ctx.save_for_backward(ids)
        ctx.rows = weight.shape[0]
        return ps.embed_rows(weight, ids)

    @staticmethod
    def backward(ctx, dout):
        ids, = ctx.saved_tensors
        return ps.embed_grad(dout.contiguous(), ids, ctx.rows), None


class Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, x, state):
        out, last = ps.gatescan(gate, x, "sigmoid", True, state=state, want_state=True)
        ctx.save_for_backward(gate, x, out, state)
        return out, last

    @staticmethod
    def backward(ctx, dout, dlast):
        gate, x, out, state = ctx.saved_tensors
        return ps.gatescan_grad(dout.contiguous(), gate, x, out, "sigmoid", True, state=state,
                                dstate_out=dlast.contiguous(), want_dstate=True)


def model(seed=0, rows=97, width=40, inner=72):
    gen = torch.Generator().manual_seed(seed)
    shapes = {"embed": (rows, width), "gate": (width, inner), "x": (width, inner)}
    return {k: (torch.randn(s, generator=gen) * 0.3).cuda() for k, s in shapes.items()}


def test_training_through_lookup_and_recurrence():
    B, T, K = 3, 150, 40
    w = model()
    gen = torch.Generator().manual_seed(1)
    ids = (97 * torch.rand((B, T), generator=gen) ** 3).long()
    ids[1, -20:] = -1                                     # a padded sequence
    state = torch.randn((B, 72), generator=gen)
    c, d = torch.randn((B, T, 72), generator=gen), torch.randn((B, 72), generator=gen)

    leaves = {k: v.clone().requires_grad_() for k, v in w.items()}
    start = state.cuda().requires_grad_()
    e = Embed.apply(leaves["embed"], ids.cuda())
    out, last = Gate.apply((e.view(-1, K) @ leaves["gate"]).view(B, T, 72), (e.view(-1, K) @ leaves["x"]).view(B, T, 72),
                           start)
    ((out * c.cuda()).sum() + (last * d.cuda()).sum()).backward()

    lens = [T] * B
    w64 = {k: v.cpu().double().numpy() for k, v in w.items()}
    flat = ids.view(-1).numpy()
    e64 = np.where((flat >= 0)[:, None], w64["embed"][flat.clip(0)], 0)
    z, x = e64 @ w64["gate"], e64 @ w64["x"]
    a, rest = ref.gates(z, "sigmoid")
    h, _ = ref.forward(a, rest * x, lens, state.numpy())
    prev = ref.before(h, lens, state.numpy())
    dh, first = ref.backward(c.view(-1, 72).double().numpy(), a, lens, d.numpy())
    dz, dx = dh * (prev - x) * a * rest, dh * rest

    mag = {k: np.abs(v) for k, v in w64.items()}
    em, xm = np.abs(e64), np.abs(e64) @ mag["x"]
    hm, _ = ref.forward(a, rest * xm, lens, state.abs().numpy())
    pm = ref.before(hm, lens, state.abs().numpy())
    dm, sm = ref.backward(c.abs().view(-1, 72).double().numpy(), a, lens, d.abs().numpy())
    zm, xg = dm * (pm + xm) * a * rest, dm * rest
    G = (em @ mag["gate"]).max()
    steps = 2 * (2 * T * (K * G + 10) + 2 * (K + 1) + B * T)

    def table(rows):
        t = np.zeros(w64["embed"].shape)
        np.add.at(t, flat[flat >= 0], rows[flat >= 0])
        return t

    def near(got, want, size):
        off = np.abs(got.detach().cpu().double().numpy().reshape(want.shape) - want)
        assert (off <= steps * U * size + 1e-30).all(), (off / (U * size + 1e-30)).max()

    near(out, h, hm)
    near(start.grad, first, sm)
    near(leaves["gate"].grad, e64.T @ dz, em.T @ zm)
    near(leaves["x"].grad, e64.T @ dx, em.T @ xg)
    near(leaves["embed"].grad, table(dz @ w64["gate"].T + dx @ w64["x"].T),
         table(zm @ mag["gate"].T + xg @ mag["x"].T))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_serving_from_prompts_to_sampled_tokens(dtype):
    """Prompts of unequal length fill a pool of states, then every step's token
    is drawn from penalized logits: call by call and as one replayed graph."""
    V, D, P, steps = 97, 40, 7, 6
    w = {k: v.to(dtype) for k, v in model(3, V, D, D).items()}
    lens = [5, 1, 130]
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    ends = torch.tensor(np.cumsum(lens), dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(4)
    prompt = torch.randint(0, V, (sum(lens),), generator=gen).cuda()
    u = torch.rand((steps, 3), generator=gen).cuda()
    mask = torch.full((2, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    mask[1, 1] = 0x0F0F0F0F
    mask_slots = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    longest = max(lens) + steps

    def project(e):
        return (e @ w["gate"]).contiguous(), (e @ w["x"]).contiguous()

    def fresh():
        pool = torch.full((P, D), 7.0, device="cuda")
        e = ps.embed_rows(w["embed"], prompt)
        h, last = ps.gatescan(*project(e), "sigmoid", True, ends=ends, want_state=True)
        pool[slots.long()] = last
        past = torch.full((3, longest), -1, dtype=torch.int32, device="cuda")
        at = 0
        for r, n in enumerate(lens):
            past[r, :n] = prompt[at:at + n].int()
            at += n
        where = torch.tensor(lens, device="cuda")
        return {"pool": pool, "past": past, "where": where, "h": h[ends.long() - 1].clone(), "u": u[0].clone(),
                "prompt": where.int(), "logits": torch.empty((3, V), dtype=dtype, device="cuda")}

    def step(s):
        s["logits"].copy_(s["h"] @ w["embed"].t())
        ps.penalize_logits(s["logits"], s["past"], prompt=s["prompt"], repetition=1.3, presence=0.4,
                           frequency=0.2, mask=mask, mask_slots=mask_slots, out=s["logits"])
        token, _, _ = ps.sample_logits(s["logits"], s["u"], temperature=0.8, top_k=20)
        s["past"].scatter_(1, s["where"][:, None], token[:, None])
        s["where"].add_(1)
        e = ps.embed_rows(w["embed"], token)
        ps.gatescan_step(*project(e), s["pool"], "sigmoid", True, slots=slots, out=s["h"])

    eager, kept = fresh(), []
    for i in range(steps):
        eager["u"].copy_(u[i])
        step(eager)
        kept.append({k: v.clone() for k, v in eager.items()})
    # the step's states and outputs are those of the whole sequences
    tokens = [torch.cat([prompt[int(e) - n:int(e)], eager["past"][r, n:n + steps].long()])
              for r, (n, e) in enumerate(zip(lens, ends.tolist()))]
    whole = ps.embed_rows(w["embed"], torch.cat(tokens))
    all_ends = torch.tensor(np.cumsum([n + steps for n in lens]), dtype=torch.int32, device="cuda")
    gate, x = project(whole)
    h, last = ps.gatescan(gate, x, "sigmoid", True, ends=all_ends, want_state=True)
    a, rest = ref.gates(gate.cpu().double().numpy(), "sigmoid")
    size = ref.forward(a, rest * np.abs(x.cpu().double().numpy()), [n + steps for n in lens])[1]
    off = (eager["pool"][slots.long()] - last).abs().cpu().double().numpy()
    # each is off by 16 u of S a token it has passed; products of other shapes
    # may round their sums of D otherwise, to the type: a gate's argument by
    # D u of its G and half a step (1/2 eps of it) on either side, and x as much
    G = (whole.abs().float() @ w["gate"].abs().float()).max().item()
    X = (whole.abs().float() @ w["x"].abs().float()).max().item()
    eps = torch.finfo(dtype).eps
    T = max(lens) + steps
    moved = 2 * (D * U + eps) * (T * G * size + T * X) if dtype != torch.float32 else 2 * D * U * T * (G * size + X)
    assert (off <= 2 * 16 * (T + 1) * U * size + moved).all()
    untouched = [i for i in range(P) if i not in slots.tolist()]
    assert bool((eager["pool"][untouched] == 7.0).all())
    drawn = eager["past"][0, lens[0]:lens[0] + steps]
    allowed = [t for t in range(V) if not 32 <= t < 64 or 0x0F0F0F0F >> (t - 32) & 1]
    assert set(drawn.tolist()) <= set(allowed)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s = fresh()
        step(s)                                           # scratch, and the products' workspaces
        first = fresh()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(s)
    for k, v in first.items():
        s[k].copy_(v)
    for i in range(steps):
        s["u"].copy_(u[i])
        graph.replay()
        torch.cuda.synchronize()
        ps.embed_rows(w["embed"], prompt)                 # eager work between replays
        for k, v in kept[i].items():
            assert torch.equal(s[k], v), (i, k)


def test_one_scratch_buffer_for_all_of_them():
    gen = torch.Generator().manual_seed(9)
    gate, x, dout = (torch.randn((2, 700, 72), generator=gen).cuda() for _ in range(3))
    wide = [torch.randn((1, 3000, 200), generator=gen).cuda() for _ in range(2)]
    ids = torch.randint(0, 5000, (9000,), generator=gen).cuda()
    rows = torch.randn((9000, 16), generator=gen).cuda()
    many = torch.randint(0, 300, (70000,), generator=gen).cuda()
    few = torch.randn((70000, 8), generator=gen).cuda()
    keys = torch.randint(0, 2 ** 31 - 1, (100001,), generator=gen).to(torch.int32).cuda()
    logits, u = torch.randn((40, 5000), generator=gen).cuda(), torch.rand(40, generator=gen).cuda()
    out, _ = ps.gatescan(gate, x, "sigmoid", True)

    def scan():
        data = keys.clone()
        ps.scan_u32_ex(data, want_total=False)
        return [data]

    calls = [
        lambda: [t for t in ps.gatescan(gate, x, "sigmoid", True, want_state=True)],
        scan,
        lambda: [ps.embed_grad(rows, ids, 5000)],
        lambda: [t for t in ps.gatescan_grad(dout, gate, x, out, "sigmoid", True, want_dstate=True)],
        lambda: [ps.radix_perm_u32(keys, 4)],
        lambda: [ps.gatescan(*wide, "sigmoid", False)[0]],
        lambda: [ps.embed_grad(few, many, 300)],
        lambda: list(ps.sample_logits(logits, u, top_k=9)),
    ]
    want = [[t.clone() for t in c()] for c in calls]
    gen = np.random.default_rng(2)
    for which in list(range(len(calls))) + gen.integers(0, len(calls), 60).tolist():
        for got, ref_ in zip(calls[which](), want[which]):
            assert torch.equal(got, ref_), which


def test_two_graphs_that_share_their_streams_scratch():
    gen = torch.Generator().manual_seed(11)
    gate, x = (torch.randn((2, 900, 72), generator=gen).cuda() for _ in range(2))
    ids = torch.randint(0, 50, (9000,), generator=gen).cuda()
    rows = torch.randn((9000, 24), generator=gen).cuda()
    jobs = [lambda: [ps.gatescan(gate, x, "sigmoid", True)[0], ps.embed_grad(rows, ids, 50)],
            lambda: [ps.embed_grad(rows[:5000], ids[:5000], 50), ps.gatescan(x, gate, "sigmoid", False)[0]]]
    want = [[t.clone() for t in j()] for j in jobs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for j in jobs:
            j()
    side.synchronize()
    graphs, outs = [], []
    for j in jobs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(j())
    with torch.cuda.stream(side):
        for which in (0, 1, 1, 0, 0, 1):
            for t in outs[which]:
                t.fill_(float("nan"))
            graphs[which].replay()
            eager = jobs[1 - which]()                     # on the graphs' stream, after it
            side.synchronize()
            for got, ref_ in zip(outs[which] + eager, want[which] + want[1 - which]):
                assert torch.equal(got, ref_)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab,length", [(3, 40001, 90000), (260, 17000, 20000)])
def test_lists_that_name_most_of_a_row(rows, vocab, length, dtype, inplace):
    """More named logits than are worked on at once, more biases than a
    workgroup's threads, in rows short of a multiple of anything.  A penalized
    logit has a product or quotient, a product with the count, and two sums, each
    off by u of the absolute values that go in, then one rounding to its type;
    f16 rounds what is below its normal numbers to half its smallest."""
    gen = torch.Generator().manual_seed(12)
    x = (torch.randn((rows, vocab), generator=gen) * 3).to(dtype)
    past = (vocab * torch.rand((1, length), generator=gen) ** 2).int().expand(rows, length).cuda()
    biased = torch.randint(-1, vocab, (1, 2500), generator=gen).int()
    values = torch.randn((1, 2500), generator=gen)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, (vocab + 31) // 32), generator=gen).int()
    slots = torch.zeros(rows, dtype=torch.int32)
    slots[::2] = -1
    prompt = torch.full((rows,), length // 3, dtype=torch.int32)
    logits = x.cuda()
    got = ps.penalize_logits(logits, past, prompt=prompt.cuda(), repetition=1.25, presence=0.5, frequency=0.25,
                             bias_tokens=biased.expand(rows, 2500).cuda(), bias_values=values.expand(rows, 2500).cuda(),
                             mask=mask.cuda(), mask_slots=slots.cuda(), out=logits if inplace else None).cpu().double()
    seen = np.bincount(past[0].cpu().numpy(), minlength=vocab) > 0
    times = np.bincount(past[0, length // 3:].cpu().numpy(), minlength=vocab)
    bias = np.zeros(vocab)
    for t, v in zip(biased[0].tolist(), values[0].tolist()):
        if t >= 0:
            bias[t] = v
    bits = np.unpackbits(mask[0].numpy().view(np.uint8), bitorder="little")[:vocab]
    y = x.double().numpy()
    scaled = np.where(seen, np.where(y > 0, y / 1.25, y * 1.25), y)
    loss = np.where(times > 0, 0.5 + 0.25 * times, 0)
    want = scaled - loss + bias
    size = np.abs(scaled) + loss + np.abs(bias)
    half = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]
    tol = half * np.abs(want) + 5 * U * size + (2.0 ** -25 if dtype == torch.float16 else 1e-37)
    shut = (bits == 0)[None, :] & (slots.numpy() == 0)[:, None]
    got = got.numpy()
    assert (got[shut] == -np.inf).all()
    assert (np.abs(got - want)[~shut] <= tol[~shut]).all()
