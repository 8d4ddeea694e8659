"""Scratch of linear attention over packed batches, without a GPU: it follows
the tokens that are cut into segments, not the number of sequences."""
import pytest

import prefix_scan_amd as ps
from prefix_scan_amd import _Shape


def need(tokens, seqs, heads, width, share=None, packed=True, dtype=1):
    sh = _Shape(dtype, seqs, heads, width, width, tokens, 0x100000 if packed else None, 0x100000, 1.0)
    if share is None:
        return ps.lib().linattn_scratch_bytes(sh)
    return ps.lib().linattn_grad_scratch_bytes(sh, heads, share, share)


@pytest.mark.parametrize("tokens, seqs", [(1 << 20, 4096), (1 << 21, 16384), (1 << 21, 1 << 20)])
def test_sequences_that_are_not_cut_take_none(tokens, seqs):
    heads, width = 32, 128
    state = heads * width * width * 4
    # a segment that is not its sequence's last holds at least 256 tokens of
    # its own, and no more of them are made than fill the GPU a few times
    assert need(tokens, seqs, heads, width) <= 1024 * width * width * 4 + state
    assert need(tokens, seqs, heads, width, share=heads) <= 1024 * width * width * 4 + 3 * state
    # partial gradients of shared heads, k's and v's
    partial = 2 * tokens * heads * width * 4
    assert need(tokens, seqs, heads, width, share=8) <= partial + 1024 * width * width * 4 + 3 * state


def test_it_does_not_grow_with_the_sequences():
    assert need(1 << 16, 1 << 15, 4, 64) <= need(1 << 16, 16, 4, 64)


@pytest.mark.parametrize("packed", [True, False])
def test_one_long_sequence_has_a_state_for_each_segment(packed):
    # 65537 tokens of 16 heads of 128: 32 segments of each, all but the last
    # with a state
    got = need(65537, 1, 16, 128, packed=packed)
    assert 31 * 16 * 128 * 128 * 4 <= got <= 33 * 16 * 128 * 128 * 4
