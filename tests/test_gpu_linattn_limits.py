"""Gradients of shared heads past 2^32 elements on the GPU."""
import pytest
import torch

import prefix_scan_amd as ps

pytestmark = pytest.mark.gpu


def test_more_elements_of_a_shared_head_than_a_grid_has_threads():
    # Two heads share k; rows that broadcast from one keep the inputs small.
    # Without memory dk(t) is scale (do(t) . v(t)) q(t), summed over the heads.
    tokens, width = (1 << 25) + 37, 128
    assert tokens * width > 1 << 32
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free memory")
    cast = lambda h, d: torch.arange(1, h * d + 1, device="cuda").view(1, 1, h, d).bfloat16() / 8  # noqa: E731
    one = lambda h, d: cast(h, d).expand(1, tokens, h, d)  # noqa: E731
    q, k, v, do = one(2, width), one(1, width), one(2, 1), one(2, 1)
    g = torch.full((2,), float("-inf"), device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        dq, dk, dv, _ = ps.linattn_grad(do, q, k, v, g, stream=stream)
    torch.cuda.synchronize()
    qh, vh, dh = (t[0, 0].double() for t in (q, v, do))
    # sums of two products of values with at most 8 bits: exact in 32 bits, rounded once
    want = (qh * (dh * vh).sum(1, keepdim=True)).sum(0).to(torch.bfloat16)
    for lo in range(0, tokens, 1 << 22):
        part = dk[0, lo:lo + (1 << 22), 0]
        assert bool((part == want).all()), lo
    del dq, dk, dv, part
    ps._scratch.pop((0, stream.cuda_stream))
    torch.cuda.empty_cache()
