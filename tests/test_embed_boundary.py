"""Embedding rows and their gradient without a GPU: the C entry points refuse
bad arguments before anything is launched, answer their size query, and do
nothing for nothing; the binding refuses bad tensors."""
import ctypes

import pytest
import torch

import prefix_scan_amd as ps
from prefix_scan_amd import _Embed

FAKE = 0x100000                        # never dereferenced: every case fails before launch
BIG = 1 << 40


def shape(**kw):
    base = dict(dtype=1, out_dtype=1, id_bytes=8, tokens=100, rows=1000, width=64, scale=1.0)
    base.update(kw)
    return _Embed(*[base[n] for n, _ in _Embed._fields_])


def rows(sh=None, weight=FAKE, ids=FAKE, out=FAKE):
    return ps.lib().embed_rows(sh or shape(), weight, 64, ids, out, 64, None)


def grad(sh=None, weight=FAKE, ids=FAKE, out=FAKE, accumulate=0, scratch=FAKE, n=BIG):
    return ps.lib().embed_grad(sh or shape(), out, 64, ids, weight, 64, accumulate, scratch, n, None)


@pytest.mark.parametrize("call", [rows, grad])
def test_arguments_are_checked(call):
    for bad in (dict(dtype=3), dict(dtype=-1), dict(out_dtype=3), dict(id_bytes=2), dict(id_bytes=0), dict(width=0)):
        assert call(shape(**bad)) == ps.ERR_ARG, bad
    for bad in (dict(rows=1 << 31), dict(tokens=(1 << 36) + 1), dict(width=(1 << 36) + 1)):
        assert call(shape(**bad)) == ps.ERR_SIZE, bad
    assert call(weight=FAKE + 1) == ps.ERR_ALIGN and call(out=FAKE + 1) == ps.ERR_ALIGN
    assert call(ids=FAKE + 4) == ps.ERR_ALIGN and call(shape(id_bytes=4), ids=FAKE + 2) == ps.ERR_ALIGN
    for name in ("weight", "ids", "out"):
        assert call(**{name: None}) == ps.ERR_NULL, name


def test_each_type_has_its_alignment():
    assert rows(shape(dtype=0), weight=FAKE + 2) == ps.ERR_ALIGN
    assert rows(shape(out_dtype=0), out=FAKE + 2) == ps.ERR_ALIGN
    assert grad(shape(dtype=0), out=FAKE + 2) == ps.ERR_ALIGN
    assert grad(shape(out_dtype=0), weight=FAKE + 2) == ps.ERR_ALIGN


def test_the_gradient_is_checked():
    assert grad(shape(tokens=1 << 31)) == ps.ERR_SIZE
    assert grad(accumulate=2) == ps.ERR_ARG
    assert grad(scratch=None) == ps.ERR_NULL
    need = ps.lib().embed_grad_scratch_bytes(shape(tokens=100000))
    # keys and positions, twice, and two rows of floats for each 128 tokens
    assert need > 16 * 100000 + 100000 // 128 * 2 * 64 * 4
    assert grad(shape(tokens=100000), n=need - 300) == ps.ERR_SCRATCH


def test_nothing_to_do():
    L = ps.lib()
    assert rows(shape(tokens=0), ids=None, out=None) == ps.OK
    assert grad(shape(rows=0), weight=None) == ps.OK
    assert grad(shape(tokens=0), accumulate=1, ids=None, out=None, scratch=None) == ps.OK
    assert L.embed_rows(None, FAKE, 64, FAKE, FAKE, 64, None) == ps.ERR_NULL
    assert L.embed_grad_scratch_bytes(None) > 0 and L.embed_grad_scratch_bytes(shape(tokens=1 << 32)) > 0


def test_the_binding_refuses():
    w, ids = torch.zeros(9, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        ps.embed_rows(w, ids)                                   # not on a GPU
    with pytest.raises(ValueError):
        ps.embed_grad(torch.zeros(3, 8), ids, 9)
    with pytest.raises(TypeError):
        ps.embed_rows(w, ids, dtype=torch.int32)
    with pytest.raises(TypeError):
        ps.embed_rows(w.int(), ids)
    with pytest.raises(TypeError):
        ps.embed_grad(w.double(), ids, 9)
    assert ctypes.sizeof(_Embed) == 48


def test_rows_that_are_evenly_spaced():
    assert ps._spaced(torch.zeros(4, 3, 8), "x") == 8
    assert ps._spaced(torch.zeros(4, 3, 16)[..., :8], "x") == 16
    assert ps._spaced(torch.zeros(4, 1, 8)[::2], "x") == 16
    assert ps._spaced(torch.zeros(8), "x") == 0 and ps._spaced(torch.zeros(1, 8), "x") == 0
    for t in (torch.zeros(4, 3, 8)[:, :2], torch.zeros(4, 3, 8).transpose(0, 1), torch.zeros(1, 3, 8).expand(4, 3, 8)):
        with pytest.raises(ValueError):
            ps._spaced(t, "x")
