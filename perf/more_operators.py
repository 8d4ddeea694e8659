"""What is measured of embedding rows, gated recurrences and penalties on logits.

`listed()` and `draw()` give cases, `prepare()` makes a case's inputs, `run()`
is one pass through an operator, in plain torch operations or (with `own`)
through this package, `work()` the bytes and operations that a pass cannot do
without, and `exact()` the outputs in 64 bits, from the operator's definition.
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_CHUNK = 128


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _scan(op, dtype, seqs, tokens, width, form, blend, ragged=0, state=True):
    return {"op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "width": width, "form": form,
            "blend": blend, "ragged": ragged, "state": state}


def _step(dtype, rows, width, form, blend, pool=0):
    return {"op": "step", "dtype": dtype, "rows": rows, "width": width, "form": form, "blend": blend, "pool": pool}


def _embed(op, dtype, vocab, width, tokens, to="", ids="int64", padded=False, scale=1.0):
    return {"op": op, "dtype": dtype, "to": to or dtype, "vocab": vocab, "width": width, "tokens": tokens,
            "ids": ids, "padded": padded, "scale": scale}


def _penalty(dtype, rows, vocab, history, packed=True, prompt=True, biases=0, grammars=0):
    return {"op": "penalty", "dtype": dtype, "rows": rows, "vocab": vocab, "history": history, "packed": packed,
            "prompt": prompt, "biases": biases, "grammars": grammars}


def listed():
    cases = {
        # one short prompt of a single user: latency
        "scan_tiny": _scan("fwd", "bf16", 1, 77, 512, "sigmoid", True),
        # an ordinary batch of training sequences
        "scan_batch": _scan("fwd", "bf16", 8, 4096, 2048, "sigmoid", True, state=False),
        # prompts of very different lengths packed one after another, some of them empty
        "scan_ragged": _scan("fwd", "fp16", 41, 500, 1000, "log", False, ragged=7),
        # one long document: few channels to work on at a time
        "scan_long": _scan("fwd", "bf16", 1, 131073, 1024, "log", True),
        # a training step's gradient over equal sequences
        "scan_train": _scan("bwd", "bf16", 8, 2048, 2560, "sigmoid", True, state=False),
        # gradients in full precision over packed documents of an odd width, with states
        "scan_train_odd": _scan("bwd", "fp32", 23, 400, 333, "decay", False, ragged=3),
        # a full server's next tokens: states of many users picked from a pool
        "scan_step": _step("bf16", 256, 4096, "sigmoid", True, pool=320),
        # a training batch's tokens to rows
        "embed_batch": _embed("embed", "bf16", 32000, 2048, 16384, scale=2048 ** 0.5),
        # their gradient, over the whole of a large table
        "embed_train": _embed("embed_grad", "bf16", 128000, 2048, 16384, scale=2048 ** 0.5),
        # packed documents with padding, a table of odd size whose gradient is kept in full precision
        "embed_train_odd": _embed("embed_grad", "fp16", 50021, 520, 9001, to="fp32", ids="int32", padded=True),
        # one user's next token: latency
        "penalty_one": _penalty("bf16", 1, 32000, 700),
        # a full server whose users each have their own settings, a few biases and grammars
        "penalty_batch": _penalty("bf16", 256, 150001, 3000, biases=12, grammars=20),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng):
    return rng.choice((64 * _spread(rng, 1, 128), 8 * _spread(rng, 1, 1024), _spread(rng, 1, 8192)))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "step", "embed", "embed_grad", "embed_grad", "penalty", "penalty"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    half = 2 if dtype == "fp32" else 1
    if op == "penalty":
        vocab = _spread(rng, 500, 200000)
        rows = _spread(rng, 1, max(1, min(512, (38000000 // half) // vocab)))
        return _penalty(dtype, rows, vocab, _spread(rng, 1, 3000), rng.random() < 0.5, rng.random() < 0.5,
                        rng.choice((0, 0, rng.randint(1, 300))), rng.choice((0, 0, rng.randint(1, 32))))
    width = _width(rng)
    if op in ("embed", "embed_grad"):
        to = rng.choice((dtype, dtype, "fp32"))
        most = (1 << 27 if to == "fp32" else 1 << 28)
        vocab = _spread(rng, 100, max(100, min(200000, most // width)))
        tokens = _spread(rng, 1, max(1, min(131072, (1 << 26) // half // width)))
        return _embed(op, dtype, vocab, width, tokens, to, rng.choice(("int32", "int64")), rng.random() < 0.5,
                      rng.choice((1.0, width ** 0.5)))
    form, blend = rng.choice(("decay", "log", "sigmoid")), rng.random() < 0.5
    if op == "step":
        rows = _spread(rng, 1, 512)
        return _step(dtype, rows, width, form, blend, rng.choice((0, rows + rng.randint(0, 64))))
    most = (1 << (26 if op == "bwd" else 27)) // half // width      # rows
    tokens = _spread(rng, 1, min(131072, most))
    seqs = _spread(rng, 1, max(1, min(64, most // tokens)))
    ragged = rng.choice((0, 0, rng.randint(1, 1 << 20))) if seqs * tokens <= 131072 else 0
    return _scan(op, dtype, seqs, tokens, width, form, blend, ragged, rng.random() < 0.5)


def _lengths(case):
    """Tokens of each sequence; where they are ragged, `tokens` is about their mean, and some
    are empty or of one token."""
    if not case["ragged"]:
        return [case["tokens"]] * case["seqs"]
    rng = random.Random(case["ragged"])
    lens = [rng.choice((0, 1, case["tokens"])) if rng.random() < 0.15
            else int(case["tokens"] * 2 * rng.random() ** 1.5) for _ in range(case["seqs"])]
    lens[0] = max(lens[0], 1)
    return lens


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

_LEAN = 2.7     # the token of rank r has a share of about 1 / (r + 2.7)


def _tokens(gen, dev, vocab, *shape):
    """Tokens as texts have them: a few often, most hardly ever."""
    u = torch.rand(shape, generator=gen, device=dev, dtype=torch.float64)
    rank = (_LEAN * (torch.exp(u * math.log((vocab + _LEAN) / _LEAN)) - 1)).long().clamp(0, vocab - 1)
    return torch.randperm(vocab, generator=gen, device=dev)[rank]


def _distinct(vocab, tokens):
    """How many tokens of `vocab` are to be expected among that many."""
    edge = np.log(np.arange(vocab + 1) + _LEAN)
    share = np.diff(edge) / (edge[-1] - edge[0])
    return int(round(float(-np.expm1(tokens * np.log1p(-np.minimum(share, 1 - 1e-12))).sum())))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape, dtype=dtype, by=1.0, at=0.0):
        return (torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * by + at).to(dtype)

    def gates(*shape):
        """Memories of one to some hundred tokens."""
        z = normal(*shape, dtype=torch.float32, by=1.5, at=2.5)
        if case["form"] == "sigmoid":
            return z.to(dtype)
        log = torch.nn.functional.logsigmoid(z)
        return (log if case["form"] == "log" else torch.exp(log)).to(dtype)

    op = case["op"]
    if op == "penalty":
        return _prepare_penalty(case, gen, dev, dtype)
    if op in ("embed", "embed_grad"):
        n, v, d = case["tokens"], case["vocab"], case["width"]
        ids = _tokens(gen, dev, v, n)
        if case["padded"]:
            ids[3::11] = -1
        s = {"op": op, "ids": ids.to(getattr(torch, case["ids"])), "scale": case["scale"], "to": _DTYPES[case["to"]]}
        if op == "embed":
            s["weight"] = normal(v, d, by=d ** -0.5)
        else:
            s.update(dout=normal(n, d), vocab=v)
        return s
    d = case["width"]
    s = {"op": op, "form": case["form"], "blend": case["blend"]}
    if op == "step":
        b, pool = case["rows"], case["pool"]
        s.update(gate=gates(b, d), x=normal(b, d), slots=None)
        s["state"] = normal(pool or b, d, dtype=torch.float32, by=2.0)
        s["state_out"] = s["state"].clone()
        if pool:      # users sit anywhere in the pool, and a row in sixteen is idle
            slots = torch.randperm(pool, generator=gen, device=dev)[:b].to(torch.int32)
            slots[3::16] = -1
            s["slots"] = slots
        return s
    lens = _lengths(case)
    b = case["seqs"]
    lead = (sum(lens),) if case["ragged"] else (b, case["tokens"])
    s.update(gate=gates(*lead, d), x=normal(*lead, d), ends=None, state=None, dstate=None)
    if case["ragged"]:
        s["ends"] = torch.tensor(np.cumsum(lens), dtype=torch.int32, device=dev)
    if case["state"]:
        s["state"] = normal(b, d, dtype=torch.float32, by=2.0)
    if op == "bwd":       # a training program has the forward pass's outputs in hand
        s["out"] = _plain_fwd(s)[0]
        s["dout"] = normal(*lead, d)
        if case["state"]:
            s["dstate"] = normal(b, d, dtype=torch.float32)
    return s


def _prepare_penalty(case, gen, dev, dtype):
    r, n, most = case["rows"], case["vocab"], case["history"]
    rand = lambda *shape: torch.rand(shape, generator=gen, device=dev)  # noqa: E731
    s = {"op": "penalty", "x": (torch.randn((r, n), generator=gen, device=dev) * 2.5).to(dtype)}
    s["out"] = torch.empty_like(s["x"])
    lens = (2 * most * rand(r)).int()                     # what users and the model have written so far
    lens[1::9] = 0
    lens[0] = most
    s["tokens"], s["ends"] = _lists(case, lens, _tokens(gen, dev, n, r, max(int(lens.max()), 1)))
    s["prompt"] = (lens * rand(r)).int() if case["prompt"] else None
    at = torch.arange(r, device=dev)
    s["repetition"] = torch.where(at % 4 == 3, 1.0, 1.0 + 0.5 * rand(r))
    s["presence"] = torch.where(at % 3 == 1, 0.0, rand(r))
    s["frequency"] = torch.where(at % 5 == 2, 0.0, 0.5 * rand(r))
    s.update(bias_tokens=None, bias_values=None, bias_ends=None, mask=None, mask_slots=None)
    if case["biases"]:
        many = torch.randint(0, case["biases"] + 1, (r,), generator=gen, device=dev)
        m = case["biases"]
        tokens = torch.randint(0, n, (r, m), generator=gen, device=dev)
        values = torch.randn((r, m), generator=gen, device=dev) * 4
        values[:, ::5] = -100.0                           # as good as banned
        s["bias_tokens"], s["bias_ends"] = _lists(case, many, tokens)
        s["bias_values"] = _lists(case, many, values)[0]
    if case["grammars"]:
        words = -(-n // 32)
        mask = torch.randint(-(1 << 31), 1 << 31, (2, case["grammars"], words), generator=gen, device=dev)
        mask = (mask[0] & mask[1]).to(torch.int32)        # a quarter of the tokens may follow
        mask[0] = 0                                       # a state that nothing follows
        s["mask"] = mask
        slots = torch.randint(0, case["grammars"], (r,), generator=gen, device=dev).to(torch.int32)
        slots[::2] = -1                                   # free text
        s["mask_slots"] = slots
    return s


def _lists(case, lens, rows):
    """A list for each row, of its first elements: (packed, their ends) or (padded with -1, None)."""
    width = rows.shape[1]
    inside = torch.arange(width, device=rows.device) < lens.view(-1, 1)
    kind = torch.float32 if rows.is_floating_point() else torch.int32
    if case["packed"]:
        return rows[inside].to(kind), torch.cumsum(lens, 0).to(torch.int32)
    return torch.where(inside, rows, -1).to(kind), None


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "embed": _plain_embed,
            "embed_grad": _plain_embed_grad, "penalty": _plain_penalty}[s["op"]](s)


def _run_own(s):
    import prefix_scan_amd as ps
    if s["op"] == "fwd":
        out, state = ps.gatescan(s["gate"], s["x"], form=s["form"], blend=s["blend"], ends=s["ends"],
                                 state=s["state"], want_state=s["state"] is not None)
        return [out] if state is None else [out, state]
    if s["op"] == "bwd":
        grads = ps.gatescan_grad(s["dout"], s["gate"], s["x"], s["out"], form=s["form"], blend=s["blend"],
                                 ends=s["ends"], state=s["state"], dstate_out=s["dstate"],
                                 want_dstate=s["state"] is not None)
        return [g for g in grads if g is not None]
    if s["op"] == "step":
        return list(ps.gatescan_step(s["gate"], s["x"], s["state"], form=s["form"], blend=s["blend"],
                                     slots=s["slots"], state_out=s["state_out"]))
    if s["op"] == "embed":
        return [ps.embed_rows(s["weight"], s["ids"], scale=s["scale"], dtype=s["to"])]
    if s["op"] == "embed_grad":
        return [ps.embed_grad(s["dout"], s["ids"], s["vocab"], scale=s["scale"], dtype=s["to"])]
    return [ps.penalize_logits(s["x"], s["tokens"], ends=s["ends"], prompt=s["prompt"],
                               repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                               bias_tokens=s["bias_tokens"], bias_values=s["bias_values"],
                               bias_ends=s["bias_ends"], mask=s["mask"], mask_slots=s["mask_slots"],
                               out=s["out"])]


def _gates(s):
    """(a, 1 - a) of the gates, in 32 bits."""
    g = s["gate"].float()
    if s["form"] == "sigmoid":
        return torch.sigmoid(g), torch.sigmoid(-g)
    if s["form"] == "log":
        return torch.exp(g), -torch.expm1(g)
    return g, 1 - g


def _runs(a, b):
    """h(t) = a(t) h(t - 1) + b(t) along the first axis, from h(-1) = 0: within chunks by steps of
    1, 2, 4, .. tokens, then over the chunks in the same way, then both together."""
    n, d = a.shape
    if n <= _CHUNK:
        return _doubled(a, b, 0)[1]
    chunks = -(-n // _CHUNK)
    pad = chunks * _CHUNK - n
    a, b = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(chunks, _CHUNK, d) for x in (a, b))
    a, b = _doubled(a, b, 1)
    last = _runs(a[:, -1].contiguous(), b[:, -1].contiguous())
    b[1:] += a[1:] * last[:-1].unsqueeze(1)
    return b.view(chunks * _CHUNK, d)[:n]


def _doubled(a, b, axis):
    n, step = a.shape[axis], 1
    while step < n:
        here = (slice(None),) * axis + (slice(step, None),)
        past = (slice(None),) * axis + (slice(None, n - step),)
        b = torch.cat([b.narrow(axis, 0, step), b[here] + a[here] * b[past]], axis)
        a = torch.cat([a.narrow(axis, 0, step), a[here] * a[past]], axis)
        step *= 2
    return a, b


def _places(s):
    """First and last token of each sequence among all rows, and which sequences have any."""
    if s["ends"] is None:
        b, t = s["gate"].shape[:2]
        first = torch.arange(b, device=s["gate"].device) * t
        return first, first + t - 1, torch.ones_like(first, dtype=torch.bool)
    ends = s["ends"].long()
    lens = torch.diff(ends, prepend=ends.new_zeros(1))
    return ends - lens, ends - 1, lens > 0


def _plain_fwd(s):
    shape, d = s["gate"].shape, s["gate"].shape[-1]
    a, rest = (x.reshape(-1, d) for x in _gates(s))
    b = s["x"].float().reshape(-1, d)
    b = rest * b if s["blend"] else b.clone()
    a = a.clone()
    first, last, live = _places(s)
    start = first[live]
    if s["state"] is not None:
        b[start] += a[start] * s["state"][live]
    a[start] = 0.0
    h = _runs(a, b)
    out = h.to(s["gate"].dtype).view(shape)
    if s["state"] is None:
        return [out]
    return [out, torch.where(live.unsqueeze(1), h[last.clamp(min=0)], s["state"])]


def _plain_bwd(s):
    d = s["gate"].shape[-1]
    flat = lambda n: s[n].float().reshape(-1, d)  # noqa: E731
    a, rest = (x.reshape(-1, d) for x in _gates(s))
    dout = flat("dout")
    first, last, live = _places(s)
    start, end = first[live], last[live]
    if s["dstate"] is not None:
        dout = dout.clone()
        dout[end] += s["dstate"][live]
    keep = a.clone()
    keep[end] = 0.0          # what comes from later tokens ends with the sequence
    g = _runs(keep.flip(0), (a * dout).flip(0)).flip(0)
    later = torch.cat([g[1:], g.new_zeros(1, d)])
    later[end] = 0.0
    dh = dout + later
    before = torch.cat([dout.new_zeros(1, d), flat("out")[:-1]])
    before[start] = 0.0 if s["state"] is None else s["state"][live]
    da = dh * (before - flat("x") if s["blend"] else before)
    dgate = {"decay": lambda: da, "log": lambda: da * a, "sigmoid": lambda: da * a * rest}[s["form"]]()
    dx = dh * rest if s["blend"] else dh
    outs = [t.to(s["gate"].dtype).view(s["gate"].shape) for t in (dgate, dx)]
    if s["state"] is None:
        return outs
    return outs + [torch.where(live.unsqueeze(1), g[first.clamp(max=len(g) - 1)], s["dstate"])]


def _plain_step(s):
    a, rest = _gates(s)
    x = s["x"].float()
    b = rest * x if s["blend"] else x
    slots = None if s["slots"] is None else s["slots"].long()
    new = a * (s["state"] if slots is None else s["state"][slots.clamp(min=0)]) + b
    if slots is None:
        s["state_out"].copy_(new)
        return [new.to(s["x"].dtype), s["state_out"]]
    live = slots >= 0
    s["state_out"][slots[live]] = new[live]
    return [torch.where(live.view(-1, 1), new, 0.0).to(s["x"].dtype), s["state_out"]]


def _plain_embed(s):
    ids = s["ids"].long()
    rows = s["weight"][ids.clamp(min=0)].float() * s["scale"]
    return [torch.where(ids.unsqueeze(1) >= 0, rows, 0.0).to(s["to"])]


def _plain_embed_grad(s):
    ids = s["ids"].long()
    sums = torch.zeros((s["vocab"] + 1, s["dout"].shape[1]), device=ids.device)
    sums.index_add_(0, torch.where(ids >= 0, ids, s["vocab"]), s["dout"].float())
    return [(sums[:-1] * s["scale"]).to(s["to"])]


def _spread_lists(tokens, ends, rows):
    """(row, place in its list, token) of every element of the rows' lists, pads left out."""
    if ends is None:
        at = torch.arange(tokens.shape[1], device=tokens.device).expand_as(tokens)
        row = torch.arange(rows, device=tokens.device).unsqueeze(1).expand_as(tokens)
        live = tokens >= 0
        return row[live], at[live], tokens[live].long(), live
    ends = ends.long()
    lens = torch.diff(ends, prepend=ends.new_zeros(1))
    row = torch.repeat_interleave(torch.arange(rows, device=tokens.device), lens, output_size=len(tokens))
    return row, torch.arange(len(tokens), device=tokens.device) - (ends - lens)[row], tokens.long(), None


def _plain_penalty(s):
    x = s["x"].float()
    r, n = x.shape
    row, at, token, _ = _spread_lists(s["tokens"], s["ends"], r)
    times = torch.zeros((2, r * n), device=x.device)
    place = row * n + token
    times[0].index_add_(0, place, torch.ones_like(place, dtype=torch.float32))
    written = torch.ones_like(place, dtype=torch.bool) if s["prompt"] is None else at >= s["prompt"][row]
    times[1].index_add_(0, place, written.float())
    seen, wrote = times.view(2, r, n)
    rep, presence, frequency = (s[k].view(r, 1) for k in ("repetition", "presence", "frequency"))
    y = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    y = y - torch.where(wrote > 0, presence + frequency * wrote, 0.0)
    if s["bias_tokens"] is not None:          # of a token that is listed twice, the last counts
        row, at, token, live = _spread_lists(s["bias_tokens"], s["bias_ends"], r)
        values = s["bias_values"] if live is None else s["bias_values"][live]
        place = row * n + token
        order = torch.full((r * n,), -1, device=x.device).scatter_reduce_(0, place, at, "amax")
        chosen = order[place] == at
        bias = torch.zeros(r * n, device=x.device)
        bias[place[chosen]] = values[chosen]
        y = y + bias.view(r, n)
    if s["mask"] is not None:
        bit = torch.arange(n, device=x.device)
        allowed = ((s["mask"][:, bit // 32] >> (bit % 32).int()) & 1) == 1
        slots = s["mask_slots"].long()
        y = torch.where(allowed[slots.clamp(min=0)] | (slots < 0).view(r, 1), y, float("-inf"))
    return [y.to(s["x"].dtype)]


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    size, op = _DTYPES[case["dtype"]].itemsize, case["op"]
    if op == "penalty":
        n = case["rows"] * case["vocab"]
        lists = case["rows"] * (4 * case["history"] + 4 * case["biases"])
        masks = min(case["grammars"], case["rows"]) * case["vocab"] // 8
        return {"bytes": 2 * n * size + lists + masks, "flops": n}
    d = case["width"]
    if op in ("embed", "embed_grad"):
        n, to = case["tokens"], _DTYPES[case["to"]].itemsize
        ids = n * (8 if case["ids"] == "int64" else 4)
        if op == "embed":
            return {"bytes": ids + n * d * to + _distinct(case["vocab"], n) * d * size, "flops": n * d}
        return {"bytes": ids + n * d * size + case["vocab"] * d * to, "flops": n * d}
    if op == "step":
        rows = case["rows"] - (len(range(3, case["rows"], 16)) if case["pool"] else 0)
        return {"bytes": rows * d * (8 + 3 * size), "flops": rows * d * 6}
    n = sum(_lengths(case)) * d
    states = case["seqs"] * d * 4 if case["state"] else 0
    if op == "fwd":
        return {"bytes": 3 * n * size + 2 * states, "flops": 6 * n}
    return {"bytes": (6 if case["blend"] else 5) * n * size + 3 * states, "flops": 12 * n}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "penalty":
        return _exact_penalty(s)
    if case["op"] in ("embed", "embed_grad"):
        return _exact_embed(case, s)
    if case["op"] == "step":
        return _exact_step(s)
    return _exact_scan(case, s)


def _exact_gates(s, gate):
    g = gate.double()
    if s["form"] == "sigmoid":
        e = torch.exp(-g.abs())
        low, high = e / (1 + e), 1 / (1 + e)
        return torch.where(g >= 0, high, low), torch.where(g >= 0, low, high)
    if s["form"] == "log":
        return torch.exp(g), -torch.expm1(g)
    return g, 1 - g


def _exact_step(s):
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device=s["x"].device)
    after = s["state"].double().clone()
    a, rest = _exact_gates(s, s["gate"])
    slots = range(len(out)) if s["slots"] is None else s["slots"].tolist()
    for row, slot in enumerate(slots):
        if slot >= 0:
            into = s["x"][row].double() * (rest[row] if s["blend"] else 1.0)
            after[slot] = a[row] * after[slot] + into
            out[row] = after[slot]
    return [out, after]


def _exact_scan(case, s):
    """Token by token, the sequences of an equal batch side by side."""
    d, dev = case["width"], s["x"].device
    if case["ragged"]:
        at, runs = 0, []
        for i, n in enumerate(_lengths(case)):
            runs.append((slice(at, at + n), slice(i, i + 1), n))
            at += n
        cut = lambda t, r: t[r[0]].unsqueeze(1)  # noqa: E731
    else:
        runs = [(None, slice(0, case["seqs"]), case["tokens"])]
        cut = lambda t, r: t.transpose(0, 1)  # noqa: E731
    names = ("out",) if case["op"] == "fwd" else ("dgate", "dx")
    outs = {n: torch.zeros(s["x"].shape, dtype=torch.float64, device=dev) for n in names}
    end = torch.zeros((case["seqs"], d), dtype=torch.float64, device=dev)
    zeros = torch.zeros((case["seqs"], d), dtype=torch.float64, device=dev)
    for r in runs:
        a, rest = _exact_gates(s, cut(s["gate"], r).contiguous())
        x = cut(s["x"], r).double().contiguous()
        first = (zeros if s["state"] is None else s["state"].double())[r[1]]
        if case["op"] == "fwd":
            b = rest * x if s["blend"] else x
            h = torch.empty_like(b)
            now = first
            for at, bt, ht in zip(a.unbind(0), b.unbind(0), h.unbind(0)):
                now = torch.addcmul(bt, at, now, out=ht)
            cut(outs["out"], r).copy_(h)
            end[r[1]] = now
            continue
        now = (zeros if s["dstate"] is None else s["dstate"].double())[r[1]].clone()
        dh = cut(s["dout"], r).double().contiguous()
        for at, dt in zip(a.unbind(0)[::-1], dh.unbind(0)[::-1]):
            dt += now
            torch.mul(at, dt, out=now)
        end[r[1]] = now
        if r[2] == 0:
            continue
        before = torch.cat([first.unsqueeze(0), cut(s["out"], r).double()[:-1]])
        slope = {"decay": 1.0, "log": a, "sigmoid": a * rest}[s["form"]]
        cut(outs["dgate"], r).copy_(dh * (before - x if s["blend"] else before) * slope)
        cut(outs["dx"], r).copy_(dh * rest if s["blend"] else dh)
    return list(outs.values()) + ([] if s["state"] is None else [end])


def _exact_embed(case, s):
    ids = s["ids"].long()
    live = (ids >= 0).nonzero().view(-1)
    if case["op"] == "embed":
        out = torch.zeros((len(ids), case["width"]), dtype=torch.float64, device=ids.device)
        for part in live.split(4096):
            out[part] = s["weight"][ids[part]].double() * s["scale"]
        return [out]
    out = torch.zeros((case["vocab"], case["width"]), dtype=torch.float64, device=ids.device)
    # The k-th time that each token is met, for k = 0, 1, ..: no token twice among them.
    mine = ids[live].cpu().numpy()
    order = np.argsort(mine, kind="stable")
    starts = np.searchsorted(mine[order], mine[order], side="left")
    met = np.empty(len(mine), dtype=np.int64)
    met[order] = np.arange(len(mine)) - starts
    by = np.argsort(met, kind="stable")
    cuts = np.cumsum(np.bincount(met)) if len(met) else []
    by = torch.from_numpy(by).to(ids.device)
    lo = 0
    for hi in cuts:
        rows = live[by[lo:int(hi)]]
        out[ids[rows]] += s["dout"][rows].double()
        lo = int(hi)
    return [out * s["scale"]]


def _exact_penalty(s):
    rows = []
    x = s["x"].double().cpu().numpy()
    host = {k: v.cpu().numpy() if isinstance(v, torch.Tensor) else v for k, v in s.items() if k not in ("x", "out")}
    n = x.shape[1]

    def part(tokens, ends, r):
        if ends is None:
            return tokens[r]
        return tokens[(ends[r - 1] if r else 0):ends[r]]

    for r in range(x.shape[0]):
        y = x[r].copy()
        past = part(host["tokens"], host["ends"], r)
        rep, presence, frequency = (float(host[k][r]) for k in ("repetition", "presence", "frequency"))
        prompt = 0 if host["prompt"] is None else int(host["prompt"][r])
        seen = np.unique(past[past >= 0])
        y[seen] = np.where(y[seen] > 0, y[seen] / rep, y[seen] * rep)
        new, times = np.unique(past[prompt:][past[prompt:] >= 0], return_counts=True)
        y[new] -= presence + frequency * times
        if host["bias_tokens"] is not None:
            given = dict(zip(part(host["bias_tokens"], host["bias_ends"], r).tolist(),
                             part(host["bias_values"], host["bias_ends"], r).tolist()))
            for token, value in given.items():
                if token >= 0:
                    y[token] += value
        if host["mask"] is not None and host["mask_slots"][r] >= 0:
            words = host["mask"][host["mask_slots"][r]].view(np.uint32)
            bits = np.unpackbits(words.view(np.uint8), bitorder="little")[:n]
            y[bits == 0] = -np.inf
        rows.append(y)
    return [np.stack(rows)]
