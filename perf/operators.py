"""What is measured of linear attention with decay and of token sampling.

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

def _attn(op, dtype, seqs, tokens, heads, dk, dv, heads_k=0, heads_v=0, ragged=0, state=True):
    return {"op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "heads": heads,
            "heads_k": heads_k or heads, "heads_v": heads_v or heads, "dk": dk, "dv": dv,
            "ragged": ragged, "state": state}


def _step(dtype, rows, heads, dk, dv, heads_k=0, heads_v=0, pool=0):
    return {"op": "step", "dtype": dtype, "rows": rows, "heads": heads,
            "heads_k": heads_k or heads, "heads_v": heads_v or heads, "dk": dk, "dv": dv,
            "pool": pool}


def _sample(dtype, rows, vocab, cut):
    return {"op": "sample", "dtype": dtype, "rows": rows, "vocab": vocab, "cut": cut}


def listed():
    cases = {
        # one short question of a single user: latency
        "prompt_tiny": _attn("fwd", "bf16", 1, 96, 4, 64, 64),
        # an ordinary batch of prompts of equal length
        "prompt_batch": _attn("fwd", "bf16", 4, 4096, 32, 128, 128, state=False),
        # prompts of very different lengths packed one after another, some of
        # them empty; keys and values shared by several heads
        "prompt_ragged": _attn("fwd", "fp16", 37, 600, 24, 72, 104, heads_k=6, heads_v=6, ragged=11),
        # one long document, with few heads to work on at a time
        "prompt_long": _attn("fwd", "bf16", 1, 65537, 16, 128, 128),
        # a training step's gradient over equal sequences
        "train_batch": _attn("bwd", "bf16", 8, 2048, 16, 128, 128, state=False),
        # gradients in full precision over packed documents, with states
        "train_odd": _attn("bwd", "fp32", 5, 700, 12, 48, 96, heads_k=4, heads_v=12, ragged=5),
        # one user's next token: latency
        "step_one": _step("bf16", 1, 16, 128, 128),
        # odd widths, shared keys, states picked from a pool
        "step_odd": _step("fp16", 19, 20, 80, 112, heads_k=5, heads_v=20, pool=40),
        # a full server: states of many users picked from a pool
        "step_batch": _step("bf16", 256, 32, 128, 128, pool=320),
        # one user's next token: latency
        "sample_one": _sample("bf16", 1, 32000, "nucleus"),
        # a decoding batch whose users each have their own settings
        "sample_batch": _sample("fp32", 48, 128000, "mixed"),
        # many samples at a time from a large vocabulary of odd size
        "sample_large": _sample("bf16", 512, 150001, "mixed"),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng, most):
    heads = rng.choice([h for h in (1, 2, 4, 6, 8, 12, 16, 20, 24, 32) if h <= most])
    shared = lambda: rng.choice([d for d in (1, 2, 3, 4, 5, 6, 8, 12, 16, 24, 32) if heads % d == 0])  # noqa: E731
    return (heads, shared(), shared()) if rng.random() < 0.4 else (heads, heads, heads)


def _width(rng):
    return rng.choice((64, 64, 128, 128, 128, rng.randint(1, 16) * 8, rng.randint(1, 128)))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "step", "sample", "sample"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "sample":
        vocab = _spread(rng, 500, 200000)
        rows = _spread(rng, 1, max(1, min(512, (36000000 if dtype == "fp32" else 72000000) // vocab)))
        return _sample(dtype, rows, vocab, rng.choice(("nucleus", "mixed", "mixed", "topk", "free")))
    heads, hk, hv = _heads(rng, 32)
    dk, dv = _width(rng), _width(rng)
    if op == "step":
        rows = _spread(rng, 1, 256)
        return _step(dtype, rows, heads, dk, dv, hk, hv, rng.choice((0, rows + rng.randint(0, 64))))
    tokens = _spread(rng, 1, 4096 if dtype == "fp32" else 16384)
    most = (1 << 28) // (tokens * heads * (dk + dv))       # the largest listed batch's elements
    most //= (2 if op == "bwd" else 1) * (2 if dtype == "fp32" else 1)
    seqs = _spread(rng, 1, max(1, min(64, most)))
    return _attn(op, dtype, seqs, tokens, heads, dk, dv, hk, hv,
                 rng.choice((0, 0, rng.randint(1, 1 << 20))), rng.random() < 0.5)


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

def _decays(heads, device):
    """The heads' memories reach from about 2^3 to 2^11 tokens."""
    at = torch.arange(heads, dtype=torch.float64) / max(heads - 1, 1)
    return torch.log1p(-torch.pow(2.0, -(3.0 + 8.0 * at))).to(torch.float32).to(device)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape, dtype=dtype, by=1.0):
        return (torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * by).to(dtype)

    if case["op"] == "sample":
        return _prepare_sample(case, gen, dev, dtype)
    h, hk, hv, dk, dv = (case[k] for k in ("heads", "heads_k", "heads_v", "dk", "dv"))
    s = {"op": case["op"], "scale": dk ** -0.5, "decay": _decays(h, dev)}
    if case["op"] == "step":
        b, pool = case["rows"], case["pool"]
        s.update(q=normal(b, h, dk), k=normal(b, hk, dk), v=normal(b, hv, dv), slots=None)
        s["state"] = normal(pool or b, h, dk, dv, dtype=torch.float32, by=3.0)
        s["state_out"] = s["state"].clone()
        if pool:      # users sit anywhere in the pool, and a row in sixteen is idle
            slots = torch.randperm(pool, generator=gen, device=dev)[:b].to(torch.int32)
            slots[3::16] = -1
            s["slots"] = slots
        return s
    lens = _lengths(case)
    b = case["seqs"]
    lead = (sum(lens),) if case["ragged"] else (b, case["tokens"])
    s.update(q=normal(*lead, h, dk), k=normal(*lead, hk, dk), v=normal(*lead, hv, dv),
             ends=None, state=None, dstate=None)
    if case["ragged"]:
        s["ends"] = torch.tensor(np.cumsum(lens), dtype=torch.int32, device=dev)
        s["longest"] = max(lens)
    if case["state"]:
        s["state"] = normal(b, h, dk, dv, dtype=torch.float32, by=3.0)
    if case["op"] == "bwd":
        s["do"] = normal(*lead, h, dv)
        if case["state"]:
            s["dstate"] = normal(b, h, dk, dv, dtype=torch.float32)
    return s


def _prepare_sample(case, gen, dev, dtype):
    r, n, cut = case["rows"], case["vocab"], case["cut"]
    rand = lambda *shape: torch.rand(shape, generator=gen, device=dev)  # noqa: E731
    x = torch.randn((r, n), generator=gen, device=dev) * 2.5
    likely = torch.randint(0, n, (r, 64), generator=gen, device=dev)      # what the model leans to
    x.scatter_add_(1, likely, -3.0 * torch.log(rand(r, 64) + 1e-3))
    x[:, 7::97] = float("-inf")                                           # tokens that a grammar bans
    if cut == "mixed" and r > 4:
        x[r // 2] = float("-inf")                                         # nothing allowed at all
    s = {"op": "sample", "x": x.to(dtype), "u": rand(r)}
    full = lambda v, t=torch.float32: torch.full((r,), v, dtype=t, device=dev)  # noqa: E731
    if cut == "nucleus":
        s.update(temperature=full(0.8), top_k=full(0, torch.int32), top_p=full(0.95), min_p=full(0.0))
    elif cut == "topk":
        s.update(temperature=full(0.7), top_k=full(40, torch.int32), top_p=full(1.0), min_p=full(0.0))
    elif cut == "free":
        s.update(temperature=full(1.0), top_k=full(0, torch.int32), top_p=full(1.0), min_p=full(0.0))
    else:
        at = torch.arange(r, device=dev)
        s["temperature"] = torch.where(at % 8 == 5, 0.0, 0.5 + rand(r))   # a user in eight: greedy
        s["top_k"] = torch.where(at % 3 == 0, 0, 1 + (rand(r) ** 3 * 1000).int()).to(torch.int32)
        s["top_p"] = torch.where(at % 4 == 1, 1.0, 0.5 + 0.5 * rand(r))
        s["min_p"] = torch.where(at % 5 == 2, 0.1 * rand(r), 0.0)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step,
            "sample": _plain_sample}[s["op"]](s)


def _run_own(s):
    import prefix_scan_amd as ps
    if s["op"] == "fwd":
        out, state = ps.linattn(s["q"], s["k"], s["v"], s["decay"], scale=s["scale"], ends=s["ends"],
                                state=s["state"], want_state=s["state"] is not None)
        return [out] if state is None else [out, state]
    if s["op"] == "bwd":
        grads = ps.linattn_grad(s["do"], s["q"], s["k"], s["v"], s["decay"], scale=s["scale"],
                                ends=s["ends"], state=s["state"], dstate_out=s["dstate"],
                                want_dstate=s["state"] is not None)
        return [g for g in grads if g is not None]
    if s["op"] == "step":
        out, state = ps.linattn_step(s["q"], s["k"], s["v"], s["decay"], s["state"], scale=s["scale"],
                                     slots=s["slots"], state_out=s["state_out"])
        return [out, state]
    return list(ps.sample_logits(s["x"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                 top_p=s["top_p"], min_p=s["min_p"]))


def _spans(s):
    """(length of each sequence [B], place of each token in a row of padded sequences or None)."""
    if s["ends"] is None:
        b, t = s["q"].shape[:2]
        return torch.full((b,), t, device=s["q"].device), None, -(-t // _CHUNK) * _CHUNK
    ends = s["ends"].long()
    lens = torch.diff(ends, prepend=ends.new_zeros(1))
    long = -(-s["longest"] // _CHUNK) * _CHUNK
    owner = torch.repeat_interleave(torch.arange(len(ends), device=ends.device), lens,
                                    output_size=s["q"].shape[0])
    at = torch.arange(s["q"].shape[0], device=ends.device) - (ends - lens)[owner]
    return lens, owner * long + at, long


def _padded(x, place, long, seqs, heads):
    """x as [B, H, long, d] in 32 bits, zeros behind each sequence, shared heads repeated."""
    x = x.float()
    if place is None:
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, long - x.shape[1]))
    else:
        x = x.new_zeros((seqs * long,) + x.shape[1:]).index_copy_(0, place, x)
        x = x.view((seqs, long) + x.shape[1:])
    return x.repeat_interleave(heads // x.shape[2], dim=2).transpose(1, 2).contiguous()


def _unpadded(x, place, tokens, heads, dtype):
    """The opposite, with the gradients of a shared head summed."""
    x = x.transpose(1, 2)
    b, t, h, d = x.shape
    x = x.reshape(b, t, heads, h // heads, d).sum(3) if heads != h else x
    x = x[:, :tokens] if place is None else x.reshape(b * t, heads, d)[place]
    return x.to(dtype).contiguous()


def _power(g, n):
    return torch.exp(g * n)


def _causal(a, b, c, g):
    """out_i = sum over j <= i of exp(g (i - j)) (a_i . b_j) c_j, by chunks: within a chunk from
    the products of its rows, from earlier chunks through their sums of b_j c_j^T."""
    B, H, T, m = a.shape
    n, C = c.shape[-1], _CHUNK
    N = T // C
    a, b, c = (x.reshape(B, H, N, C, x.shape[-1]) for x in (a, b, c))
    g = g.view(1, H, 1, 1, 1)
    at = torch.arange(C, device=a.device, dtype=torch.float32)
    ahead = at.view(C, 1) - at.view(1, C)
    near = torch.where(ahead >= 0, _power(g, ahead.clamp(min=0)), 0.0)
    out = ((a @ b.transpose(-1, -2).contiguous()) * near) @ c
    sums = (b * _power(g, C - 1 - at.view(C, 1))).transpose(-1, -2).contiguous() @ c
    step = torch.arange(N, device=a.device, dtype=torch.float32)
    back = step.view(N, 1) - 1 - step.view(1, N)
    far = torch.where(back >= 0, _power(g.view(1, H, 1, 1), C * back.clamp(min=0)), 0.0)
    before = (far @ sums.reshape(B, H, N, m * n)).view(B, H, N, m, n)
    return (out + (a * _power(g, at.view(C, 1) + 1)) @ before).reshape(B, H, T, n)


def _ages(s, lens, long):
    """exp(g (t + 1)), and exp(g (len - 1 - t)) inside each sequence: [B, H, long, 1] each."""
    t = torch.arange(long, device=lens.device, dtype=torch.float32)
    g = s["decay"].view(1, -1, 1)
    left = lens.view(-1, 1, 1) - 1 - t
    after = torch.where(left >= 0, _power(g, left.clamp(min=0)), 0.0)
    return _power(g, t + 1).unsqueeze(-1), after.unsqueeze(-1)


def _whole(s, lens):
    return _power(s["decay"].view(1, -1), lens.view(-1, 1))[..., None, None]


def _plain_fwd(s):
    lens, place, long = _spans(s)
    h = s["q"].shape[-2]
    q, k, v = (_padded(s[n], place, long, len(lens), h) for n in ("q", "k", "v"))
    out = _causal(q, k, v, s["decay"])
    if s["state"] is None:
        return [_unpadded(out * s["scale"], place, s["q"].shape[1], h, s["q"].dtype)]
    since, after = _ages(s, lens, long)
    out = (out + (q * since) @ s["state"]) * s["scale"]
    state = _whole(s, lens) * s["state"] + (k * after).transpose(-1, -2).contiguous() @ v
    return [_unpadded(out, place, s["q"].shape[1], h, s["q"].dtype), state]


def _plain_bwd(s):
    lens, place, long = _spans(s)
    h = s["q"].shape[-2]
    q, k, v, do = (_padded(s[n], place, long, len(lens), h) for n in ("q", "k", "v", "do"))
    q = q * s["scale"]
    back = lambda *xs: _causal(*(x.flip(2) for x in xs), s["decay"]).flip(2)  # noqa: E731
    dq = _causal(do, v, k, s["decay"])
    dk = back(v, do, q)
    dv = back(k, q, do)
    dstate = None
    if s["state"] is not None:
        since, after = _ages(s, lens, long)
        dq = dq + (do * since) @ s["state"].transpose(-1, -2).contiguous()
        dk = dk + (v * after) @ s["dstate"].transpose(-1, -2).contiguous()
        dv = dv + (k * after) @ s["dstate"]
        dstate = _whole(s, lens) * s["dstate"] + (q * since).transpose(-1, -2).contiguous() @ do
    grads = [_unpadded(x, place, s["q"].shape[1], s[n].shape[-2], s[n].dtype)
             for x, n in ((dq * s["scale"], "q"), (dk, "k"), (dv, "v"))]
    return grads if dstate is None else grads + [dstate]


def _plain_step(s):
    q, k, v, state = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
    h = q.shape[1]
    k, v = (x.repeat_interleave(h // x.shape[1], dim=1) for x in (k, v))
    g = torch.exp(s["decay"]).view(1, h, 1, 1)
    slots = None if s["slots"] is None else s["slots"].long()
    old = state if slots is None else state[slots.clamp(min=0)]
    new = old * g + k.unsqueeze(-1) * v.unsqueeze(-2)
    out = (q.unsqueeze(-2) @ new).squeeze(-2) * s["scale"]
    if slots is None:
        s["state_out"].copy_(new)
        return [out.to(s["q"].dtype), s["state_out"]]
    live = slots >= 0
    s["state_out"][slots[live]] = new[live]
    return [torch.where(live.view(-1, 1, 1), out, 0.0).to(s["q"].dtype), s["state_out"]]


def _plain_sample(s):
    x = s["x"].double()
    r, n = x.shape
    dev = x.device
    cut = {k: s[k].double().view(r, 1) for k in ("temperature", "top_p", "min_p", "u")}
    x = torch.where(torch.isnan(x), float("-inf"), x)
    top = x.amax(1, keepdim=True)
    empty = torch.isneginf(top)
    greedy = cut["temperature"] <= 0
    w = torch.exp((x - torch.where(empty, 0.0, top)) / torch.where(greedy, 1.0, cut["temperature"]))
    down, order = torch.sort(x, dim=1, descending=True, stable=True)
    wd = w.gather(1, order)
    rank = torch.arange(n, device=dev).view(1, n)
    k = torch.where(s["top_k"] > 0, s["top_k"].long(), n).view(r, 1)
    keep = (rank < k) & (wd >= cut["min_p"].clamp(max=1.0)) & ~torch.isneginf(down)
    sums = torch.cumsum(torch.where(keep, wd, 0.0), 1)
    before = sums - torch.where(keep, wd, 0.0)
    nucleus = (cut["top_p"] >= 1) | (rank == 0) | (before < cut["top_p"] * sums[:, -1:])
    keep &= torch.where(greedy, rank == 0, nucleus)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    run_ = torch.cumsum(torch.where(kept, w, 0.0), 1)
    total = run_[:, -1:]
    token = torch.argmax((run_ > cut["u"] * total).int(), 1, keepdim=True)
    logprob = torch.log(torch.where(greedy, 1.0, w.gather(1, token) / total))
    return [torch.where(empty, -1, token).view(r).int(),
            torch.where(empty, float("-inf"), logprob).view(r).float(),
            keep.sum(1).int()]


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        size = _DTYPES[case["dtype"]].itemsize
        return {"bytes": n * size + case["rows"] * 32, "flops": 4 * n}
    h, hk, hv, dk, dv = (case[k] for k in ("heads", "heads_k", "heads_v", "dk", "dv"))
    size = _DTYPES[case["dtype"]].itemsize
    if case["op"] == "step":
        rows = case["rows"] - (len(range(3, case["rows"], 16)) if case["pool"] else 0)
        return {"bytes": rows * h * dk * dv * 8 + rows * size * (h * dk + hk * dk + hv * dv + h * dv),
                "flops": rows * h * dk * dv * 4}
    n = sum(_lengths(case))
    states = case["seqs"] * h * dk * dv * 4 if case["state"] else 0
    inputs = h * dk + hk * dk + hv * dv
    if case["op"] == "fwd":
        return {"bytes": n * size * (inputs + h * dv) + 2 * states, "flops": n * h * dk * dv * 4}
    return {"bytes": n * size * (2 * inputs + h * dv) + 3 * states, "flops": n * h * dk * dv * 10}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "step":
        return _exact_step(s)
    return _exact_attn(case, s)


def _exact_step(s):
    out = torch.zeros(s["q"].shape[:2] + s["v"].shape[2:], dtype=torch.float64, device=s["q"].device)
    after = s["state"].double().clone()
    lam = torch.exp(s["decay"].double())
    b, h = s["q"].shape[:2]
    slots = list(range(b)) if s["slots"] is None else s["slots"].tolist()
    gk, gv = h // s["k"].shape[1], h // s["v"].shape[1]
    ik = torch.arange(h, device=out.device) // gk
    iv = torch.arange(h, device=out.device) // gv
    for row, slot in enumerate(slots):
        if slot < 0:
            continue
        kv = s["k"][row, ik].double()[:, :, None] * s["v"][row, iv].double()[:, None, :]
        after[slot] = after[slot] * lam[:, None, None] + kv
        out[row] = (s["q"][row].double()[:, :, None] * after[slot]).sum(1) * s["scale"]
    return [out, after]


def _exact_attn(case, s):
    """Each output from the pairs of tokens it sums over, one head of one sequence and one block
    of rows at a time."""
    h = case["heads"]
    names = ["q", "k", "v"] + (["do"] if case["op"] == "bwd" else [])
    lens = _lengths(case)
    dev = s["q"].device
    flat = {n: s[n].reshape((-1,) + s[n].shape[-2:]) for n in names}
    shape = lambda n, like: torch.zeros(like.shape[:-2] + (h, like.shape[-1]), dtype=torch.float64, device=dev)  # noqa: E731
    fwd = case["op"] == "fwd"
    first = [shape(n, flat[n]) for n in (["v"] if fwd else names[:3])]
    state = None
    if s["state"] is not None:
        state = torch.zeros(s["state"].shape, dtype=torch.float64, device=dev)
    scale, block, at = s["scale"], 2048, 0
    for b, length in enumerate(lens):
        for i in range(h):
            g = s["decay"][i].double()
            one = {n: flat[n][at:at + length, i // (h // flat[n].shape[1])].double() for n in names}
            t = torch.arange(length, dtype=torch.float64, device=dev)
            got = [f[at:at + length, i] for f in first]
            for lo in range(0, length, block):
                hi = min(lo + block, length)
                # rows lo..hi against the columns they reach
                gap = t[lo:hi, None] - t[None, :hi]
                near = torch.where(gap >= 0, torch.exp(g * gap), 0.0)
                if fwd:
                    got[0][lo:hi] = scale * (((one["q"][lo:hi] @ one["k"][:hi].T) * near) @ one["v"][:hi])
                    continue
                pairs = scale * near * (one["do"][lo:hi] @ one["v"][:hi].T)
                got[0][lo:hi] = pairs @ one["k"][:hi]
                got[1][:hi] += pairs.T @ one["q"][lo:hi]
                got[2][:hi] += (scale * near * (one["q"][lo:hi] @ one["k"][:hi].T)).T @ one["do"][lo:hi]
            if state is None:
                continue
            since = torch.exp(g * (t + 1))[:, None]
            left = torch.exp(g * (length - 1 - t))[:, None]
            s0 = s["state"][b, i].double()
            gone = torch.exp(g * length)
            if fwd:
                got[0] += scale * since * (one["q"] @ s0)
                state[b, i] = gone * s0 + (one["k"] * left).T @ one["v"]
                continue
            ds = s["dstate"][b, i].double()
            got[0] += scale * since * (one["do"] @ s0.T)
            got[1] += left * (one["v"] @ ds.T)
            got[2] += left * (one["k"] @ ds)
            state[b, i] = gone * ds + scale * (one["q"] * since).T @ one["do"]
        at += length
    outs = []
    for f, n in zip(first, ["q"] if fwd else names[:3]):
        heads = h if fwd else s[n].shape[-2]
        f = f.view(f.shape[0], heads, h // heads, f.shape[-1]).sum(2)
        outs.append(f.view(s[n].shape[:-2] + f.shape[1:]))
    return outs if state is None else outs + [state]


def _exact_sample(s):
    tokens, logs, kepts = [], [], []
    for r in range(s["x"].shape[0]):
        x = s["x"][r].double()
        u, temp, top_p, min_p = (float(s[n][r].double()) for n in ("u", "temperature", "top_p", "min_p"))
        top_k = int(s["top_k"][r])
        live = (x > float("-inf")).nonzero().view(-1)
        if live.numel() == 0:
            tokens.append(-1), logs.append(float("-inf")), kepts.append(0)
            continue
        best = live[x[live].argmax()] if live.numel() else None
        top = float(x[best])
        if temp <= 0:
            tokens.append(int((x == top).nonzero()[0])), logs.append(0.0), kepts.append(1)
            continue
        w = torch.exp((x[live] - top) / temp)
        order = torch.argsort(-x[live], stable=True).cpu().numpy()
        if top_k > 0:
            order = order[:top_k]
        wd = w.cpu().numpy()[order]
        held = int((wd >= min(min_p, 1.0)).sum())
        wd = wd[:held]
        if top_p < 1:
            sums = np.cumsum(wd)
            held = max(1, int(np.searchsorted(sums, top_p * sums[-1], side="left")) + 1)
        keep = np.sort(order[:held])
        mine = w.cpu().numpy()[keep]
        run_ = np.cumsum(mine)
        j = min(int(np.searchsorted(run_, u * run_[-1], side="right")), len(keep) - 1)
        tokens.append(int(live[int(keep[j])])), kepts.append(len(keep))
        logs.append(math.log(mine[j] / run_[-1]))
    return [np.asarray(tokens, dtype=np.int32), np.asarray(logs), np.asarray(kepts, dtype=np.int32)]
