"""Sampling on the GPU against its definition in 64 bits: tokens and counts
are equal, log-probabilities within half a float's step of their own and
what 64-bit sums leave (2^-24 of them and 2^-40)."""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def check(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """x: [R, V] on the host; the settings are numbers or arrays of R."""
    rows = x.shape[0]
    dev = lambda v, t: torch.as_tensor(v, dtype=t).cuda() if np.ndim(v) else v  # noqa: E731
    u = np.asarray(u, np.float32)
    out = [torch.full((rows,), -7, dtype=torch.int32).cuda(), torch.full((rows,), 7.0).cuda(),
           torch.full((rows,), -7, dtype=torch.int32).cuda()]
    ps.sample_logits(x.cuda(), torch.from_numpy(u).cuda(), dev(temperature, torch.float32),
                     dev(top_k, torch.int32), dev(top_p, torch.float32), dev(min_p, torch.float32),
                     tokens=out[0], logprobs=out[1], kept=out[2])
    token, logprob, kept = (t.cpu().numpy() for t in out)
    values = x.double().numpy()
    at = lambda v, r: np.float32(v[r] if np.ndim(v) else v)  # noqa: E731
    for r in range(rows):
        want = ref.sample(values[r], u[r], at(temperature, r), int(at(top_k, r)), at(top_p, r), at(min_p, r))
        assert (token[r], kept[r]) == (want[0], want[2]), "row %d: %s, not %s" % (
            r, (token[r], logprob[r], kept[r]), want)
        if np.isfinite(want[1]):
            assert abs(logprob[r] - want[1]) <= 2.0 ** -24 * abs(want[1]) + 2.0 ** -40, r
        else:
            assert logprob[r] == want[1], r


def logits(rows, vocab, dtype, seed=0, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, vocab), generator=gen) * spread).to(DTYPES[dtype])


def uniform(rows, seed=1):
    return np.random.default_rng(seed).random(rows, dtype=np.float32)


SETTINGS = [{}, {"temperature": 0.0}, {"temperature": 0.3, "top_k": 40}, {"top_p": 0.9},
            {"min_p": 0.05}, {"top_k": 1}, {"temperature": 5.0, "top_k": 500, "top_p": 0.5},
            {"temperature": 1.3, "top_k": 100, "top_p": 0.95, "min_p": 0.02}, {"top_p": 0.0},
            {"top_k": 7, "min_p": 1.0}, {"temperature": 100.0, "top_p": 0.999}]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 1000, 4097, 50001, 140000])
def test_sizes_and_settings(vocab, dtype):
    rows = 5 if vocab > 40000 else 9
    x = logits(rows, vocab, dtype, vocab)
    for i, s in enumerate(SETTINGS):
        check(x, uniform(rows, i), **s)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [1, 2, 300])
def test_each_row_has_its_own_settings(rows, dtype):
    rng = np.random.default_rng(rows)
    x = logits(rows, 3001, dtype, 5)
    check(x, uniform(rows), rng.choice([0.0, 0.5, 1.0, 2.0], rows).astype(np.float32),
          rng.integers(-1, 60, rows).astype(np.int32),
          rng.choice([0.1, 0.8, 0.99, 1.0, 2.0], rows).astype(np.float32),
          rng.choice([0.0, 0.01, 0.5], rows).astype(np.float32))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_equal_logits_go_by_index(dtype):
    x = torch.zeros((6, 1500), dtype=DTYPES[dtype])
    x[1, ::2] = -0.0                       # the zeros are one value
    x[2, 700:] = 1.0
    x[3] = torch.arange(1500) % 4
    x[4, 3::5] = -1.0
    for s in ({}, {"top_k": 10}, {"top_k": 801}, {"top_p": 0.5}, {"top_p": 0.25, "top_k": 700},
              {"min_p": 0.5}, {"temperature": 0.0}):
        for u in (0.0, 0.37, 0.99999994):
            check(x, np.full(6, u), **s)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_masked_rows(dtype):
    inf = float("inf")
    x = logits(8, 2000, dtype, 3)
    x[0] = -inf
    x[1] = float("nan")
    x[2, :] = -inf
    x[2, 1999] = -30.0                     # one token left, the last
    x[3, ::2] = -inf
    x[4, ::3] = float("nan")
    x[5] = torch.finfo(DTYPES[dtype]).min  # a mask of the lowest value, everywhere
    x[6] = torch.finfo(DTYPES[dtype]).min
    x[6, 77] = 2.0
    x[7, [5, 900]] = inf
    for s in SETTINGS:
        check(x, uniform(8, 4), **s)


def test_the_ends_of_u():
    x = logits(4, 5000, "fp32", 6)
    for u in (0.0, 2.0 ** -24, 1.0 - 2.0 ** -24, 1.0, 5.0, -1.0, float("nan")):
        check(x, np.full(4, u), top_p=0.9)
        check(x, np.full(4, u))


def test_strided_rows():
    x = logits(7, 1003, "bf16", 8)
    wide = torch.full((7, 1203), 50.0, dtype=torch.bfloat16).cuda()
    view = wide[:, 101:1104]
    view.copy_(x)
    u = torch.from_numpy(uniform(7)).cuda()
    a = ps.sample_logits(view, u, top_k=20, top_p=0.9)
    b = ps.sample_logits(x.cuda(), u, top_k=20, top_p=0.9)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_nothing_to_do():
    u = torch.empty(0, device="cuda")
    assert ps.sample_logits(torch.empty(0, 50, device="cuda"), u)[0].shape == (0,)
    t, logprob, kept = ps.sample_logits(torch.empty(2, 0, device="cuda"), torch.zeros(2, device="cuda"))
    assert t.tolist() == [-1, -1] and kept.tolist() == [0, 0] and torch.isneginf(logprob).all()


def test_captured_and_replayed_on_another_stream():
    x = logits(33, 20011, "fp32", 9).cuda()
    u = torch.from_numpy(uniform(33)).cuda()
    outs = [torch.empty(33, dtype=t, device="cuda") for t in (torch.int32, torch.float32, torch.int32)]
    call = lambda: ps.sample_logits(x, u, 0.8, 50, 0.9, 0.01, *outs)  # noqa: E731
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for rep in range(4):
        x.copy_(logits(33, 20011, "fp32", 20 + rep))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(-7)
        with torch.cuda.stream(stream):
            ps.scan_exclusive_u32(torch.arange(100000, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), rep


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_cuts_among_thousands_of_equal_logits(dtype):
    # More tokens in the cut's bin, or under top_k, than a list holds.
    x = torch.zeros((4, 20011), dtype=DTYPES[dtype])
    x[1, ::2] = 1.0
    x[2] = (torch.arange(20011) % 7).to(DTYPES[dtype]) / 1024        # inside the first bin
    x[3] = logits(1, 20011, dtype, 11)[0]
    for s in ({"top_k": 9999}, {"top_p": 0.5}, {"top_k": 15000, "top_p": 0.75}, {"top_k": 20010},
              {"top_k": 12000, "top_p": 0.25, "min_p": 0.3}, {"top_p": 0.9999, "temperature": 50.0}):
        for u in (0.0, 0.61, 0.99999994):
            check(x, np.full(4, u), **s)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_scales_of_logits(dtype):
    # All logits within one step of another, and spread over the type's range.
    gen = torch.Generator().manual_seed(12)
    base = torch.randn((5, 9001), generator=gen)
    x = torch.stack([base[0] * 1e-4, base[1] * 0.01 + 100.0, base[2] * 5000.0, base[3] * 1e-30,
                     base[4].exp() * 3]).to(DTYPES[dtype])
    for s in ({}, {"top_p": 0.9}, {"top_k": 50, "top_p": 0.8}, {"temperature": 1e-3, "top_p": 0.9},
              {"temperature": 3e38, "top_p": 0.5}, {"temperature": 1e-38, "top_p": 0.9}):
        check(x, uniform(5, 13), **s)


@pytest.mark.parametrize("rows", [5, 700])
def test_rows_that_start_anywhere(rows):
    for dtype in DTYPES:
        for vocab in (37, 1021):
            x = logits(rows, vocab, dtype, 14)
            u = torch.from_numpy(uniform(rows)).cuda()
            want = ps.sample_logits(x.cuda(), u, 0.9, 30, 0.95)
            for stride, at in ((vocab + 1, 1), (vocab + 3, 2), (2 * vocab + 5, 5)):
                flat = torch.full((rows * stride + 8,), 60.0, dtype=DTYPES[dtype], device="cuda")
                view = flat[at:at + rows * stride].view(rows, stride)[:, :vocab]
                view.copy_(x)
                got = ps.sample_logits(view, u, 0.9, 30, 0.95)
                assert all(torch.equal(a, b) for a, b in zip(got, want)), (dtype, vocab, stride)


def test_a_large_vocabulary():
    n = (1 << 24) - 3
    gen = torch.Generator(device="cuda").manual_seed(15)
    x = (torch.randn((1, n), generator=gen, device="cuda") * 2).bfloat16()
    for s in ({}, {"top_p": 0.9}, {"top_k": 100}, {"min_p": 0.01}):
        check(x.cpu(), uniform(1, 16), **s)
