"""Embedding rows and their gradient on the GPU against the definition in 64
bits.

Tolerances.  A rounding to a type moves a value by at most eps / 2 of it.  A
row of the lookup is scaled in 32 bits (2^-24 of it) and rounded once.  A sum of
k rows takes k additions and at most 8 more where chunks are joined, each off
by 2^-24 of the sum S of the absolute values, and so are its scaling and the
addition to what was there; f16 rounds what is below its normal numbers to
half its smallest.
"""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25, torch.float32: 1e-37}


def randn(*shape, dtype=torch.float32, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def skewed(n, rows, seed=0):
    """A few ids often, most hardly ever."""
    u = torch.rand(n, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    return (rows * u ** 4).long().clamp(max=max(rows - 1, 0))


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("to", list(DTYPES))
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("width", [1, 3, 8, 65, 520, 2050])
def test_lookup(width, dtype, to, kind):
    weight = randn(211, width, dtype=DTYPES[dtype])
    ids = skewed(301, 211)
    ids[::7], ids[5], ids[6] = -1, 211, 2 ** 31 - 1
    out = torch.full((301, width), float("nan"), dtype=DTYPES[to], device="cuda")
    got = ps.embed_rows(weight.cuda(), ids.to(kind).cuda(), 1.7, out=out)
    assert got is out
    live = (ids >= 0) & (ids < 211)
    want = torch.where(live[:, None], weight[ids.clamp(0, 210)].double() * float(np.float32(1.7)), 0.0)
    off = (got.cpu().double() - want).abs()
    assert bool((off <= (HALF[DTYPES[to]] + 2.0 ** -23) * want.abs() + TINY[DTYPES[to]]).all())
    if to == dtype:
        same = ps.embed_rows(weight.cuda(), ids.to(kind).cuda()).cpu()
        assert torch.equal(same, torch.where(live[:, None], weight[ids.clamp(0, 210)], torch.zeros((), dtype=same.dtype)))


def test_lookup_shapes_and_strides():
    weight = randn(50, 24, dtype=torch.bfloat16).cuda()
    wide = torch.zeros(50, 31, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:27] = weight
    ids = skewed(60, 50).cuda()
    want = weight[ids]
    assert torch.equal(ps.embed_rows(wide[:, 3:27], ids), want)
    assert torch.equal(ps.embed_rows(weight, ids.view(5, 4, 3)), want.view(5, 4, 3, 24))
    assert torch.equal(ps.embed_rows(weight, ids[7]), want[7])
    out = torch.full((60, 41), 7.0, dtype=torch.bfloat16, device="cuda")
    ps.embed_rows(weight, ids, out=out[:, 5:29])
    assert torch.equal(out[:, 5:29], want) and bool((out[:, :5] == 7).all()) and bool((out[:, 29:] == 7).all())
    assert ps.embed_rows(weight, ids[:0]).shape == (0, 24)
    assert not ps.embed_rows(weight[:0], ids).any()
    huge = torch.tensor([2 ** 40, -2 ** 40, 3, 2 ** 32 + 3], device="cuda")
    assert torch.equal(ps.embed_rows(weight, huge)[2], weight[3]) and not ps.embed_rows(weight, huge)[[0, 1, 3]].any()


def check(n, rows, width, dtype="fp32", to="fp32", ids=None, kind=torch.int64, scale=0.7, accumulate=False,
          strided=False):
    """The gradient; a dense one starts as NaN."""
    ids = skewed(n, rows) if ids is None else ids
    dout = randn(n, width, dtype=DTYPES[dtype], seed=1)
    live = (ids >= 0) & (ids < rows)
    dev = dout.cuda()
    dev[~live.cuda()] = float("nan")                     # rows that are not to be read
    old = randn(rows, width, dtype=DTYPES[to], seed=2)
    held = old.cuda() if accumulate else torch.full((rows, width), float("nan"), dtype=DTYPES[to], device="cuda")
    if strided:
        a = torch.full((n, width + 3), float("nan"), dtype=dev.dtype, device="cuda")
        a[:, 1:1 + width] = dev
        b = torch.full((rows, width + 5), 7.0, dtype=held.dtype, device="cuda")
        b[:, 3:3 + width] = held
        dev, held = a[:, 1:1 + width], b[:, 3:3 + width]
    got = ps.embed_grad(dev, ids.to(kind).cuda(), rows, scale, dweight=held, accumulate=accumulate)
    assert got is held
    if strided:
        assert bool((b[:, :3] == 7).all()) and bool((b[:, 3 + width:] == 7).all())
    s = float(np.float32(scale))
    at, d = ids[live], dout[live].double()
    want = torch.zeros(rows, width, dtype=torch.float64).index_add_(0, at, d) * s
    size = torch.zeros(rows, width, dtype=torch.float64).index_add_(0, at, d.abs()) * s
    if accumulate:
        want, size = want + old.double(), size + old.double().abs()
    k = torch.bincount(at, minlength=rows).double()[:, None]
    off = (got.cpu().double() - want).abs()
    tol = HALF[DTYPES[to]] * want.abs() + (k + 11) * 2.0 ** -24 * size + TINY[DTYPES[to]]
    assert bool(torch.isfinite(got).all())
    assert bool((off <= tol).all()), (off - tol).max()
    return got


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 63, 65, 511, 4095, 4096, 4097, 9001])
@pytest.mark.parametrize("rows", [1, 2, 300, 513, 20000])
def test_counts(n, rows):
    check(n, rows, 20)


@pytest.mark.parametrize("n,rows", [(50, 3), (5000, 70), (9000, 300000), (4500, 1 << 20), (600, (1 << 18) + 1)])
@pytest.mark.parametrize("dtype,to", [(d, t) for d in DTYPES for t in DTYPES])
def test_types(n, rows, dtype, to):
    check(n, rows, 8, dtype, to, kind=torch.int32 if n % 100 else torch.int64)


@pytest.mark.parametrize("width", [1, 3, 64, 65, 256, 520, 2050])
def test_widths(width):
    check(777, 100, width, "bf16", "bf16")
    check(5001, 40, width, "fp16", "fp32", accumulate=True)


def test_many_tokens():
    # more tiles than a workgroup adds up by itself; two passes and three
    check(600000, 3000, 4)
    check(600000, 1 << 19, 1, "bf16", "fp32")


@pytest.mark.parametrize("n", [700, 9000])
def test_a_table_of_many_rows(n):
    # four passes
    rows = (1 << 27) + 5
    ids = torch.randint(0, rows, (n,), generator=torch.Generator().manual_seed(4))
    ids[::5], ids[7] = rows - 1, 0
    dout = randn(n, 2) + 3.0
    got = ps.embed_grad(dout.cuda(), ids.cuda(), rows)
    used, at = ids.unique(return_inverse=True)
    want = torch.zeros(len(used), 2, dtype=torch.float64).index_add_(0, at, dout.double())
    size = torch.zeros(len(used), 2, dtype=torch.float64).index_add_(0, at, dout.double().abs())
    assert int((got != 0).any(1).sum()) == len(used)
    assert bool(((got[used.cuda()].cpu().double() - want).abs() <= (n + 11) * 2.0 ** -24 * size).all())


@pytest.mark.parametrize("accumulate", [False, True])
def test_one_id_for_all(accumulate):
    for n in (40, 4000, 70000):
        check(n, 17, 24, "bf16", "fp32", torch.full((n,), 11), accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [30, 6000])
def test_ids_that_are_no_rows(n, accumulate):
    ids = skewed(n, 90)
    ids[::3], ids[1], ids[4], ids[7] = -1, 90, 2 ** 40, -2 ** 40
    check(n, 90, 33, ids=ids, accumulate=accumulate)
    none = torch.full((n,), -1)
    check(n, 90, 33, ids=none, accumulate=accumulate)
    small = ids.clamp(-5, 95)
    check(n, 90, 33, ids=small, kind=torch.int32, accumulate=accumulate)


@pytest.mark.parametrize("edge", [8, 16, 128])
def test_runs_that_end_with_their_chunks(edge):
    # each id's run begins or ends next to a chunk's border
    n = 512 * edge
    for shift in (-1, 0, 1):
        ids = ((torch.arange(n) + shift) // edge).clamp(min=0)
        check(n, n // edge + 1, 8, ids=ids[torch.randperm(n, generator=torch.Generator().manual_seed(3))])
        check(n, n // edge + 1, 8, ids=ids // 3)


@pytest.mark.parametrize("accumulate", [False, True])
def test_strides(accumulate):
    check(900, 100, 40, "bf16", "bf16", strided=True, accumulate=accumulate)
    check(9000, 1000, 33, "fp16", "fp32", strided=True, accumulate=accumulate)


def test_nothing():
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    dout = torch.zeros(0, 24, device="cuda")
    assert not ps.embed_grad(dout, ids, 1000).any()
    held = torch.ones(1000, 24, device="cuda")
    assert bool((ps.embed_grad(dout, ids, 1000, dweight=held, accumulate=True) == 1).all())
    assert not ps.embed_grad(dout, ids, 1000, dweight=held).any()
    assert ps.embed_grad(dout, ids, 0).shape == (0, 24)
    assert ps.embed_grad(torch.ones(5, 24, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda"), 0).shape == (0, 24)


def test_shapes():
    ids = skewed(60, 9).cuda()
    dout = randn(60, 16).cuda()
    want = ps.embed_grad(dout, ids, 9)
    assert torch.equal(ps.embed_grad(dout.view(5, 12, 16), ids.view(5, 12), 9), want)
    one = ps.embed_grad(dout[3], ids[3], 9)
    assert torch.equal(one[ids[3]], dout[3]) and int((one != 0).any(1).sum()) == 1
    half = ps.embed_grad(dout, ids, 9, dtype=torch.bfloat16)
    assert half.dtype == torch.bfloat16 and torch.equal(half, want.bfloat16())


def test_the_same_bits_every_time():
    ids, dout = skewed(70000, 500).cuda(), randn(70000, 64, dtype=torch.bfloat16).cuda()
    want = ps.embed_grad(dout, ids, 500, dtype=torch.float32)
    for _ in range(8):
        assert torch.equal(ps.embed_grad(dout, ids, 500, dtype=torch.float32), want)


@pytest.mark.parametrize("n", [900, 30000])
def test_captured_and_replayed(n):
    ids, dout = skewed(n, 3000).cuda(), randn(n, 72, dtype=torch.bfloat16).cuda()
    weight = randn(3000, 72, dtype=torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [ps.embed_grad(dout, ids, 3000, 2.0).clone(), ps.embed_rows(weight, ids, 2.0).clone()]
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = [ps.embed_grad(dout, ids, 3000, 2.0), ps.embed_rows(weight, ids, 2.0)]
        for i in range(4):
            for t in got:
                t.fill_(float("nan"))
            ps.scan_exclusive_u32(torch.ones(200000, dtype=torch.int32, device="cuda"))
            ps.embed_grad(dout[:400 + i], ids[:400 + i], 100)
            graph.replay()
            side.synchronize()
            for g, w in zip(got, want):
                assert torch.equal(g, w)


def test_on_another_stream():
    ids, dout = skewed(30000, 3000).cuda(), randn(30000, 72).cuda()
    want = ps.embed_grad(dout, ids, 3000), ps.embed_rows(dout, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ps.embed_grad(dout, ids, 3000, stream=side), ps.embed_rows(dout, ids, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_as_autograds_forward_and_backward():
    weight = randn(40, 16).cuda().requires_grad_()
    ids = skewed(100, 40).cuda().view(4, 25)
    with pytest.raises(RuntimeError, match="gradient"):
        ps.embed_rows(weight, ids)

    class Embed(torch.autograd.Function):
        @staticmethod
        def forward(ctx, weight, ids):
            ctx.save_for_backward(ids)
            ctx.rows = weight.shape[0]
            return ps.embed_rows(weight, ids, 3.0)

        @staticmethod
        def backward(ctx, dout):
            return ps.embed_grad(dout.contiguous(), *ctx.saved_tensors, ctx.rows, 3.0), None

    Embed.apply(weight, ids).square().sum().backward()
    plain = weight.detach().double().requires_grad_()
    (3.0 * plain[ids]).square().sum().backward()
    assert torch.allclose(weight.grad.double(), plain.grad, rtol=1e-5, atol=1e-5)
