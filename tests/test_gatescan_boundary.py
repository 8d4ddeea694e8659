"""The gated recurrence without a GPU: the C entry points refuse bad arguments
before anything is launched, answer their size queries, and do nothing for
nothing; the binding refuses bad tensors."""
import ctypes

import pytest
import torch

import prefix_scan_amd as ps
from prefix_scan_amd import _GateRows, _GateShape

FAKE = 0x100000                        # never dereferenced: every case fails before launch
BIG = 1 << 30


def shape(**kw):
    base = dict(dtype=1, form=2, blend=1, clear_rest=0, seqs=2, tokens=100, width=64, ends=None)
    base.update(kw)
    return _GateShape(*[base[n] for n, _ in _GateShape._fields_])


def rows(data=FAKE):
    return _GateRows(data, 6400, 64)


def fwd(sh=None, gate=None, x=None, out=None, state=None, state_out=None, scratch=FAKE, n=BIG):
    return ps.lib().gatescan(sh or shape(), gate or rows(), x or rows(), state, out or rows(), state_out, scratch,
                             n, None)


def bwd(sh=None, state=None, dstate_out=None, dstate=None, scratch=FAKE, n=BIG, **kw):
    r = [kw.get(name) or rows() for name in ("dout", "gate", "x", "out", "dgate", "dx")]
    return ps.lib().gatescan_grad(sh or shape(), *r[:4], state, dstate_out, *r[4:], dstate, scratch, n, None)


def step(sh=None, gate=None, x=None, out=None, state=FAKE, pool=2, slots=None, state_out=FAKE):
    return ps.lib().gatescan_step(sh or shape(), gate or rows(), x or rows(), state, pool, slots, out or rows(),
                                  state_out, None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_shapes_are_checked(call):
    for bad in (dict(dtype=3), dict(dtype=-1), dict(form=3), dict(form=-1), dict(blend=2), dict(clear_rest=2),
                dict(width=0)):
        assert call(shape(**bad)) == ps.ERR_ARG, bad
    for bad in (dict(seqs=(1 << 24) + 1), dict(tokens=(1 << 36) + 1), dict(width=(1 << 36) + 1)):
        assert call(shape(**bad)) == ps.ERR_SIZE, bad
    assert call(shape(ends=FAKE + 2)) == ps.ERR_ALIGN
    assert call(gate=rows(FAKE + 1)) == ps.ERR_ALIGN and call(shape(dtype=0), x=rows(FAKE + 2)) == ps.ERR_ALIGN
    assert call(gate=rows(None)) == ps.ERR_NULL and call(x=rows(None)) == ps.ERR_NULL
    assert call(out=rows(None)) == ps.ERR_NULL


@pytest.mark.parametrize("call", [fwd, bwd])
def test_what_no_grid_holds_is_refused(call):
    for bad in (dict(tokens=1 << 31, width=1), dict(seqs=1 << 24, width=64, tokens=1),
                dict(width=1 << 30, tokens=1), dict(tokens=1 << 30, width=1 << 10, ends=FAKE)):
        assert call(shape(**bad)) == ps.ERR_SIZE, bad
        assert ps.lib().gatescan_scratch_bytes(shape(**bad), 0) < 1 << 12


def test_forward_is_checked():
    L = ps.lib()
    assert fwd(state=FAKE + 2) == ps.ERR_ALIGN and fwd(state_out=FAKE + 1) == ps.ERR_ALIGN
    assert fwd(state=FAKE, state_out=FAKE) == ps.ERR_ARG
    assert fwd(scratch=None) == ps.ERR_NULL
    big = shape(tokens=1 << 16)
    need = L.gatescan_scratch_bytes(big, 0)
    assert need > 1 << 16 and fwd(big, n=need - 300) == ps.ERR_SCRATCH
    assert L.gatescan(None, rows(), rows(), None, rows(), None, FAKE, BIG, None) == ps.ERR_NULL
    assert L.gatescan(shape(), rows(), None, None, rows(), None, FAKE, BIG, None) == ps.ERR_NULL
    assert fwd(shape(seqs=0), rows(None), rows(None), rows(None), scratch=None, n=0) == ps.OK


def test_gradient_is_checked():
    L = ps.lib()
    for name in ("dout", "dgate", "dx"):
        assert bwd(**{name: rows(None)}) == ps.ERR_NULL
        assert bwd(**{name: rows(FAKE + 1)}) == ps.ERR_ALIGN
    for name in ("state", "dstate_out", "dstate"):
        assert bwd(**{name: FAKE + 2}) == ps.ERR_ALIGN
    assert bwd(dstate=FAKE, dstate_out=FAKE) == ps.ERR_ARG and bwd(dstate=FAKE, state=FAKE) == ps.ERR_ARG
    assert bwd(scratch=None) == ps.ERR_NULL
    big = shape(tokens=1 << 16)
    assert bwd(big, n=L.gatescan_scratch_bytes(big, 1) - 300) == ps.ERR_SCRATCH
    # x is looked at with blend only
    r = rows()
    assert L.gatescan_grad(shape(), r, r, None, r, None, None, r, r, None, FAKE, BIG, None) == ps.ERR_NULL
    assert L.gatescan_grad(shape(blend=0), r, r, None, r, None, None, r, r, None, FAKE, 0, None) == ps.ERR_SCRATCH
    assert bwd(shape(seqs=0), scratch=None, n=0) == ps.OK


def test_step_is_checked():
    assert step(state=None) == ps.ERR_NULL and step(state_out=None) == ps.ERR_NULL
    assert step(slots=FAKE + 2) == ps.ERR_ALIGN and step(state=FAKE + 2) == ps.ERR_ALIGN
    assert step(pool=(1 << 36) + 1) == ps.ERR_SIZE
    assert step(shape(seqs=0), state=None, state_out=None) == ps.OK


def test_the_binding_refuses():
    x = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError):
        ps.gatescan(x, x)                                       # not on a GPU
    with pytest.raises(ValueError):
        ps.gatescan_grad(x, x, x, x)
    with pytest.raises(ValueError):
        ps.gatescan_step(x[:, 0], x[:, 0], torch.zeros(2, 8))
    with pytest.raises(TypeError):
        ps.gatescan(x.int(), x)
    with pytest.raises(ValueError, match="form"):
        ps.gatescan(x, x, form="exp")
    for call in (lambda: ps.gatescan(x, None), lambda: ps.gatescan_grad(x, x, None, x, blend=True),
                 lambda: ps.gatescan_grad(None, x, x, x), lambda: ps.gatescan_grad(x, x, x, None),
                 lambda: ps.gatescan_step(x[:, 0], None, x[:, 0])):
        with pytest.raises(TypeError):
            call()


def test_structures_match_the_header():
    assert ctypes.sizeof(_GateRows) == 24 and ctypes.sizeof(_GateShape) == 48
