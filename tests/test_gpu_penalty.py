"""Penalties, biases and masks on logits on the GPU against the definition in
64 bits.

Tolerances.  A logit takes at most five roundings of 32 bits -- the quotient or
product, presence + frequency * g (one), the difference, the bias's sum and the
parameters' own products -- each of 2^-24 of a value no larger than the sum S
of the absolute values, and one to the type (eps / 2 of it).  What nothing
touches keeps its bits.
"""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def host(t):
    return None if t is None else t.detach().cpu().numpy()


def part(tokens, ends, r):
    if ends is None:
        return tokens[r]
    return tokens[ends[r - 1] if r else 0:ends[r]]


def define(x, tokens=None, ends=None, prompt=None, repetition=1.0, presence=0.0, frequency=0.0, bias_tokens=None,
           bias_values=None, bias_ends=None, mask=None, mask_slots=None):
    """(what comes out in 64 bits, S, which logits are touched)."""
    y = x.double().cpu().numpy()
    size, touched = np.abs(y), np.zeros(y.shape, dtype=bool)
    n = y.shape[1]
    each = [np.broadcast_to(np.float32(v) if not torch.is_tensor(v) else host(v), (len(y),)).astype(np.float64)
            for v in (repetition, presence, frequency)]
    tokens, ends, prompt, bias_tokens, bias_values, bias_ends, mask, mask_slots = (
        host(t) for t in (tokens, ends, prompt, bias_tokens, bias_values, bias_ends, mask, mask_slots))
    for r in range(len(y)):
        rep, pres, freq = (v[r] for v in each)
        rep = rep if rep > 0 else 1.0
        pres, freq = (0.0 if np.isnan(v) else v for v in (pres, freq))
        if tokens is not None:
            past = part(tokens, ends, r)
            ok = lambda t: t[(t >= 0) & (t < n)]  # noqa: E731
            seen = np.unique(ok(past))
            touched[r, seen] = True
            with np.errstate(invalid="ignore"):
                y[r, seen] = np.where(y[r, seen] > 0, y[r, seen] / rep, y[r, seen] * rep)
            new, g = np.unique(ok(past[max(0 if prompt is None else int(prompt[r]), 0):]), return_counts=True)
            size[r, seen] = np.abs(y[r, seen])
            y[r, new] -= pres + freq * g
            size[r, new] += np.abs(pres) + np.abs(freq) * g
        if bias_tokens is not None:
            given = dict(zip(part(bias_tokens, bias_ends, r).tolist(), part(bias_values, bias_ends, r).tolist()))
            for t, v in given.items():
                if 0 <= t < n:
                    y[r, t] += v
                    size[r, t] += abs(v)
                    touched[r, t] = True
        if mask is not None:
            slot = r if mask_slots is None else mask_slots[r]
            if 0 <= slot < len(mask):
                bits = np.unpackbits(mask[slot].view(np.uint32).view(np.uint8), bitorder="little")[:n]
                y[r, bits == 0] = -np.inf
                touched[r, bits == 0] = True
    return y, size, touched


def check(x, dtype, places=("new", "out", "here"), **kw):
    want, size, touched = define(x, **kw)
    dev = {k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()}
    for place in places:
        given = x.cuda()
        out = {"new": None, "out": torch.full_like(given, 77.0), "here": given}[place]
        got = ps.penalize_logits(given, out=out, **dev)
        assert (out is None or got is out) and (place == "here" or torch.equal(given.cpu().nan_to_num(5), x.nan_to_num(5)))
        got = got.cpu()
        raw = torch.int32 if dtype == "fp32" else torch.int16
        still = torch.from_numpy(~touched)
        assert torch.equal(got.view(raw)[still], x.view(raw)[still]), place
        g = got.double().numpy()
        fixed = ~np.isfinite(want)
        assert np.array_equal(g[fixed], want[fixed], equal_nan=True), place
        with np.errstate(invalid="ignore"):
            tol = HALF[dtype] * np.abs(want) + 6 * 2.0 ** -24 * size + (2.0 ** -25 if dtype == "fp16" else 1e-37)
            off = np.abs(g - want)
        assert (off[~fixed] <= tol[~fixed]).all(), place


def case(rows, vocab, longest, dtype, packed, prompt=True, biases=0, grammars=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=gen)  # noqa: E731
    x = (torch.randn((rows, vocab), generator=gen) * 3).to(DTYPES[dtype])
    ints = lambda high, *s: torch.randint(0, max(high, 1), s, generator=gen)  # noqa: E731
    kw = {}

    def lists(most, name):
        lens = ints(most + 1, rows)
        lens[0], lens[rows // 2] = most, 0
        t = (vocab * rand(rows, max(most, 1)) ** 3).int()
        t[rand(rows, max(most, 1)) < 0.05] = -1
        t[rand(rows, max(most, 1)) < 0.02] = vocab
        inside = torch.arange(t.shape[1]) < lens[:, None]
        if packed:
            return t[inside], torch.cumsum(lens, 0).int(), inside
        return torch.where(inside, t, -1).int(), None, inside

    kw["tokens"], kw["ends"], _ = lists(longest, "tokens")
    if prompt:
        kw["prompt"] = ints(longest + 3, rows).int() - 1
    kw["repetition"], kw["presence"], kw["frequency"] = 0.5 + rand(rows), rand(rows) - 0.3, rand(rows) - 0.3
    kw["repetition"][::3] = 1.0
    if biases:
        kw["bias_tokens"], kw["bias_ends"], inside = lists(biases, "bias")
        values = torch.randn(inside.shape, generator=gen) * 5
        kw["bias_values"] = values[inside] if packed else values
    if grammars:
        kw["mask"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (grammars, (vocab + 31) // 32), generator=gen).int()
        kw["mask"][0] = 0
        kw["mask_slots"] = ints(grammars + 2, rows).int() - 1
    return x, kw


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,vocab,longest", [(1, 1, 3), (1, 7, 0), (2, 33, 40), (3, 2047, 300), (5, 2049, 1),
                                                (4, 4097, 1025), (1, 32000, 700), (40, 30001, 90)])
def test_penalties(rows, vocab, longest, dtype, packed):
    x, kw = case(rows, vocab, longest, dtype, packed, prompt=rows != 3)
    check(x, dtype, **kw)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,vocab", [(1, 5), (3, 100), (7, 4096), (6, 9003), (50, 90001)])
def test_biases_and_masks(rows, vocab, dtype, packed):
    x, kw = case(rows, vocab, 60, dtype, packed, biases=40, grammars=4)
    check(x, dtype, **kw)
    check(x, dtype, places=("out",), **{k: v for k, v in kw.items() if k.startswith("bias")})
    check(x, dtype, places=("out", "here"), **{k: v for k, v in kw.items() if k.startswith("mask")})


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_numbers_for_all_rows(dtype):
    x, kw = case(4, 500, 50, dtype, False)
    check(x, dtype, tokens=kw["tokens"], repetition=1.3, presence=0.4, frequency=0.1)
    check(x, dtype, tokens=kw["tokens"], repetition=1.3)
    check(x, dtype)


@pytest.mark.parametrize("off", [0.0, -1.0, float("nan")])
def test_what_is_off(off):
    x, kw = case(3, 300, 20, "fp32", False)
    nan = float("nan")
    check(x, "fp32", tokens=kw["tokens"], repetition=off, presence=nan, frequency=nan)
    full = lambda v: torch.full((3,), v)  # noqa: E731
    check(x, "fp32", tokens=kw["tokens"], repetition=full(off), presence=full(nan), frequency=full(0.2))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_logits_that_are_not_finite(dtype):
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[inf, -inf, nan, 1.0, -1.0, 0.0, -0.0, inf, -inf, nan, 2.0]]).to(DTYPES[dtype])
    tokens = torch.tensor([[0, 1, 2, 3, 4, 5, 6, 0]], dtype=torch.int32)
    check(x, dtype, tokens=tokens, repetition=1.5, presence=0.5, frequency=0.25)
    check(x, dtype, tokens=tokens, repetition=1.5, bias_tokens=torch.tensor([[3, 4, 3, 7]], dtype=torch.int32),
          bias_values=torch.tensor([[9.0, -inf, 1.0, 2.0]]))
    check(x, dtype, mask=torch.tensor([[0b01010101010]], dtype=torch.int32))


def test_a_token_listed_often():
    # one token many times, and a bias list whose last entry for it counts
    x = torch.randn(2, 5000)
    tokens = torch.full((2, 30000), 4321, dtype=torch.int32)
    tokens[1, ::2] = 17
    check(x, "fp32", tokens=tokens, presence=0.5, frequency=0.001, prompt=torch.tensor([10000, 0], dtype=torch.int32))
    values = torch.arange(3000.0).view(1, -1).repeat(2, 1)
    check(x, "fp32", bias_tokens=torch.full((2, 3000), 4999, dtype=torch.int32), bias_values=values)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strides(dtype):
    x, kw = case(5, 1001, 40, dtype, False, biases=9, grammars=3)
    wide = torch.full((5, 1100), 7.0, dtype=x.dtype, device="cuda")
    wide[:, 3:1004] = x.cuda()
    far = torch.full((5, 1200), 7.0, dtype=x.dtype, device="cuda")
    spread = torch.full((5, 60), 3, dtype=torch.int32, device="cuda")
    spread[:, 2:42] = kw["tokens"].cuda()
    dev = {k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()}
    want = ps.penalize_logits(x.cuda(), **dev)
    dev["tokens"] = spread[:, 2:42]
    got = ps.penalize_logits(wide[:, 3:1004], out=far[:, 5:1006], **dev)
    assert torch.equal(got, want) and bool((far[:, :5] == 7).all()) and bool((far[:, 1006:] == 7).all())
    ps.penalize_logits(wide[:, 3:1004], out=wide[:, 3:1004], **dev)
    assert torch.equal(wide[:, 3:1004], want) and bool((wide[:, :3] == 7).all()) and bool((wide[:, 1004:] == 7).all())


def test_one_list_and_mask_for_all_rows():
    x = torch.randn(4, 300)
    one = torch.tensor([[5, 9, 5]], dtype=torch.int32)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, 10)).int()
    kw = dict(tokens=one.expand(4, 3), frequency=0.5, bias_tokens=one.expand(4, 3),
              bias_values=torch.tensor([[1.0, 2.0, 3.0]]).expand(4, 3), mask=mask.expand(4, 10))
    want, size, _ = define(x, **{k: v.contiguous() if torch.is_tensor(v) else v for k, v in kw.items()})
    lists = {k: v[:1].cuda().expand(4, -1) if torch.is_tensor(v) else v for k, v in kw.items()}
    got = ps.penalize_logits(x.cuda(), **lists).cpu().double().numpy()
    finite = np.isfinite(want)
    assert np.array_equal(finite, np.isfinite(got))
    assert (np.abs(got[finite] - want[finite]) <= 8 * 2.0 ** -24 * size[finite]).all()


def test_ends_past_the_list_stay_in_it():
    x = torch.randn(3, 200, device="cuda")
    tokens = torch.arange(10, dtype=torch.int32, device="cuda")
    for ends in ([4, 500, 20], [10, 4, 10], [-1, -1, -1]):
        got = ps.penalize_logits(x, tokens, torch.tensor(ends, dtype=torch.int32, device="cuda"), presence=1.0)
        assert torch.equal(got[:, 10:], x[:, 10:])


def test_nothing():
    for shape in ((0, 50), (5, 0)):
        assert ps.penalize_logits(torch.zeros(shape, device="cuda")).shape == shape
    with pytest.raises(RuntimeError, match="gradient"):
        ps.penalize_logits(torch.zeros(2, 5, device="cuda", requires_grad=True))


def test_captured_and_on_another_stream():
    x, kw = case(6, 5000, 100, "bf16", True, biases=5, grammars=3)
    dev = {k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()}
    given = x.cuda()
    want = ps.penalize_logits(given, **dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ps.penalize_logits(given, stream=side, **dev)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = ps.penalize_logits(given, **dev)
    for _ in range(3):
        got.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
