"""The flag that may be or-ed to a type, without a GPU."""
import pytest

import prefix_scan_amd as ps
from tests.test_linattn_boundary import FAKE, bwd, fwd, rows, shape, step

FLAG = 0x100


@pytest.mark.parametrize("call", [fwd, bwd])
def test_it_changes_no_check(call):
    for dtype in (0, 1, 2):
        for kw in (dict(), dict(ends=FAKE)):
            assert call(shape(dtype=dtype | FLAG, **kw), n=0) == ps.ERR_SCRATCH
            assert call(shape(dtype=dtype | FLAG, heads=0, **kw)) == ps.ERR_ARG
    assert call(shape(dtype=0 | FLAG), q=rows(data=FAKE + 2)) == ps.ERR_ALIGN
    for bad in (3 | FLAG, 1 | 2 * FLAG, 1 | 3 * FLAG, -1, -FLAG):
        assert call(shape(dtype=bad)) == ps.ERR_ARG, bad
    assert call(shape(dtype=1 | FLAG, ends=FAKE, seqs=0), n=0) == ps.OK


def test_scratch_is_the_same():
    L = ps.lib()
    for kw in (dict(tokens=1 << 20), dict(tokens=1 << 20, ends=FAKE)):
        a, b = shape(**kw), shape(dtype=1 | FLAG, **kw)
        assert L.linattn_scratch_bytes(a) == L.linattn_scratch_bytes(b) > 1 << 16
        assert L.linattn_grad_scratch_bytes(a, 4, 2, 1) == L.linattn_grad_scratch_bytes(b, 4, 2, 1) > 1 << 16


def test_single_tokens_have_none():
    assert step(shape(dtype=1 | FLAG)) == ps.ERR_ARG
