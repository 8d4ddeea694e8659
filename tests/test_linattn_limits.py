"""Sizes that no grid covers are refused before anything is launched, without
a GPU.  A grid has fewer than 2^32 threads along each side."""
import pytest

import prefix_scan_amd as ps
from tests.test_linattn_boundary import bwd, fwd, rows, shape, step


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("ends", [None, 0x100000])
def test_too_many_sequences(call, ends):
    # a workgroup a sequence: 512 threads where a width is above 64, else 256
    wide, narrow = 1 << 23, 1 << 24
    assert call(shape(seqs=wide, tokens=1, key_width=65, ends=ends)) == ps.ERR_SIZE
    assert call(shape(seqs=wide + 1, tokens=1, value_width=128, ends=ends)) == ps.ERR_SIZE
    assert call(shape(seqs=narrow, tokens=1, ends=ends)) == ps.ERR_SIZE
    # the last that fit are refused for their scratch alone
    for sh in (shape(seqs=wide - 1, tokens=1, key_width=65, ends=ends),
               shape(seqs=narrow - 1, tokens=1, ends=ends)):
        assert call(sh, n=0) == ps.ERR_SCRATCH


def test_too_many_rows_of_a_step():
    # 256 threads a row
    assert step(shape(seqs=1 << 24), pool=1 << 24) == ps.ERR_SIZE
    # the last that fit pass the checks of sizes: no log_decay is found next
    assert step(shape(seqs=(1 << 24) - 1, log_decay=None), pool=1 << 24) == ps.ERR_NULL
