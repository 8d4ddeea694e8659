"""The gated recurrence over batches of 128 lines of tiles and more, whose
looks back span fewer tiles, with shares of the lines that differ from counter
to counter; against the definition in 64 bits, with the tolerances derived
where `near` is defined."""
import pytest
import torch

import prefix_scan_amd as ps
from tests.test_gpu_gatescan import DTYPES, check, make

pytestmark = pytest.mark.gpu

# Channels of a line.
SIDE = {"bf16": 64, "fp16": 64, "fp32": 32}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("form,blend", [("sigmoid", True), ("log", False), ("decay", True)])
@pytest.mark.parametrize("seqs,lines,cut", [(19, 7, 0), (20, 8, 3), (43, 3, 8), (149, 1, 0)])
def test_equal_sequences(seqs, lines, cut, form, blend, dtype):
    assert seqs * lines >= 128
    check((900,) * seqs, lines * SIDE[dtype] - cut, dtype, form, blend, packed=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", [(1500,), (1100, 0, 2, 700, 1, 0, 129, 256)])
def test_packed(lens, dtype):
    check(lens, 129 * SIDE[dtype] - 5, dtype, "sigmoid", True)
    check(lens, 131 * SIDE[dtype], dtype, "log", False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lines", [127, 128, 129, 257])
def test_the_same_bits_every_time(lines, dtype):
    width = lines * SIDE[dtype]
    s = make((2500,), width, dtype, "sigmoid", state=False)
    gate, x, dout = (s[k].cuda()[None] for k in ("gate", "x", "dout"))
    out, last = ps.gatescan(gate, x, "sigmoid", True, want_state=True)
    grads = ps.gatescan_grad(dout, gate, x, out, "sigmoid", True, want_dstate=True)
    # each line by itself: the same tiles, and so the same bits, with other lines about it
    few = slice(0, 2 * SIDE[dtype])
    alone, alast = ps.gatescan(gate[..., few], x[..., few], "sigmoid", True, want_state=True)
    assert torch.equal(alone, out[..., few]) and torch.equal(alast, last[:, few])
    for _ in range(4):
        again = ps.gatescan(gate, x, "sigmoid", True, want_state=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], last)
        for g, w in zip(ps.gatescan_grad(dout, gate, x, out, "sigmoid", True, want_dstate=True), grads):
            assert torch.equal(g, w)
