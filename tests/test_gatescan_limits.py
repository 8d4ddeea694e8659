"""The largest gated recurrences that are taken, as libscan.h states them:
fewer than 2^24 tiles of 128 tokens, 256 of f32's forward pass, by 64 channels,
32 of f32.  No GPU: what is taken fails for want of scratch."""
import pytest

import prefix_scan_amd as ps
from tests.test_gatescan_boundary import FAKE, bwd, fwd, shape

MOST = (1 << 24) - 1


@pytest.mark.parametrize("call,dtype,tokens,channels", [(fwd, 0, 256, 32), (fwd, 1, 128, 64), (fwd, 2, 128, 64),
                                                        (bwd, 0, 128, 32), (bwd, 1, 128, 64), (bwd, 2, 128, 64)])
def test_tiles(call, dtype, tokens, channels):
    size = lambda **kw: call(shape(dtype=dtype, **kw), n=0)  # noqa: E731
    for seqs, ends in ((1, None), (3, FAKE)):
        assert size(seqs=seqs, ends=ends, tokens=MOST * tokens, width=1) == ps.ERR_SCRATCH
        assert size(seqs=seqs, ends=ends, tokens=MOST * tokens + 1, width=1) == ps.ERR_SIZE
    assert size(seqs=1, tokens=5 * tokens, width=MOST // 5 * channels) == ps.ERR_SCRATCH
    assert size(seqs=1, tokens=5 * tokens, width=(MOST // 5 + 1) * channels) == ps.ERR_SIZE
    assert size(seqs=MOST // 3, tokens=2 * tokens + 1, width=7) == ps.ERR_SCRATCH
    assert size(seqs=MOST // 3 + 1, tokens=2 * tokens + 1, width=7) == ps.ERR_SIZE


def test_sequences():
    assert fwd(shape(seqs=1 << 24, ends=FAKE), n=0) == ps.ERR_SCRATCH
    assert fwd(shape(seqs=(1 << 24) + 1, ends=FAKE), n=0) == ps.ERR_SIZE
    assert fwd(shape(seqs=MOST, tokens=1), n=0) == ps.ERR_SCRATCH and fwd(shape(seqs=MOST + 1, tokens=1), n=0) == ps.ERR_SIZE
