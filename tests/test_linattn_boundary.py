"""Linear attention and sampling without a GPU: the C entry points refuse bad
arguments before anything is launched, answer their size queries, and do
nothing for nothing; the binding refuses bad tensors."""
import ctypes

import pytest
import torch

import prefix_scan_amd as ps
from prefix_scan_amd import _Rows, _Sample, _Shape

FAKE = 0x100000                        # never dereferenced: every case fails before launch
BIG = 1 << 30


def shape(**kw):
    base = dict(dtype=1, seqs=2, heads=4, key_width=64, value_width=64, tokens=100, ends=None,
                log_decay=FAKE, scale=1.0)
    base.update(kw)
    return _Shape(*[base[n] for n, _ in _Shape._fields_])


def rows(heads=4, data=FAKE, width=64):
    return _Rows(data, 100 * heads * width, heads * width, width, heads)


def fwd(sh=None, q=None, k=None, v=None, out=None, state=None, state_out=None, scratch=FAKE, n=BIG):
    return ps.lib().linattn(sh or shape(), q or rows(), k or rows(), v or rows(), state, out or rows(),
                            state_out, scratch, n, None)


def bwd(sh=None, state=None, dstate_out=None, dstate=None, scratch=FAKE, n=BIG, **kw):
    r = [kw.get(name) or rows() for name in ("dout", "q", "k", "v", "dq", "dk", "dv")]
    return ps.lib().linattn_grad(sh or shape(), *r[:4], state, dstate_out, *r[4:], dstate, scratch, n,
                                 None)


def step(sh=None, q=None, k=None, v=None, out=None, state=FAKE, pool=2, slots=None, state_out=FAKE):
    return ps.lib().linattn_step(sh or shape(), q or rows(), k or rows(), v or rows(), state, pool, slots,
                                 out or rows(), state_out, None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_shapes_are_checked(call):
    for bad in (dict(dtype=3), dict(dtype=-1), dict(heads=0), dict(key_width=0), dict(value_width=0),
                dict(key_width=129), dict(value_width=129)):
        assert call(shape(**bad)) == ps.ERR_ARG, bad
    for bad in (dict(heads=65536), dict(seqs=(1 << 24) + 1), dict(tokens=(1 << 36) + 1)):
        assert call(shape(**bad)) == ps.ERR_SIZE, bad
    for bad in (dict(ends=FAKE + 2), dict(log_decay=FAKE + 1)):
        assert call(shape(**bad)) == ps.ERR_ALIGN, bad
    assert call(shape(log_decay=None)) == ps.ERR_NULL
    # three heads do not divide four; more heads than the operator has
    assert call(k=rows(3)) == ps.ERR_ARG and call(v=rows(8)) == ps.ERR_ARG and call(q=rows(0)) == ps.ERR_ARG
    assert call(q=rows(data=FAKE + 1)) == ps.ERR_ALIGN
    assert call(shape(dtype=0), k=rows(data=FAKE + 2)) == ps.ERR_ALIGN
    assert call(v=rows(data=None)) == ps.ERR_NULL


def test_forward_is_checked():
    L = ps.lib()
    assert fwd(out=rows(2)) == ps.ERR_ARG                     # an output has every head
    assert fwd(out=rows(data=None)) == ps.ERR_NULL
    assert fwd(state=FAKE + 2) == ps.ERR_ALIGN and fwd(state_out=FAKE + 1) == ps.ERR_ALIGN
    assert fwd(state=FAKE, state_out=FAKE) == ps.ERR_ARG
    assert fwd(scratch=None) == ps.ERR_NULL
    big = shape(tokens=1 << 20)
    need = L.linattn_scratch_bytes(big)
    assert need > 0 and fwd(big, n=need - 300) == ps.ERR_SCRATCH
    assert L.linattn(None, rows(), rows(), rows(), None, rows(), None, FAKE, BIG, None) == ps.ERR_NULL
    # nothing to do
    assert fwd(shape(seqs=0, log_decay=None), rows(data=None), rows(data=None), rows(data=None),
               rows(data=None), scratch=None, n=0) == ps.OK


def test_gradient_is_checked():
    L = ps.lib()
    assert bwd(dout=rows(2)) == ps.ERR_ARG
    assert bwd(dk=rows(2)) == ps.ERR_ARG                      # as many heads as k
    assert bwd(dv=rows(data=None)) == ps.ERR_NULL
    for name in ("state", "dstate_out", "dstate"):
        assert bwd(**{name: FAKE + 2}) == ps.ERR_ALIGN
    assert bwd(dstate=FAKE, dstate_out=FAKE) == ps.ERR_ARG and bwd(dstate=FAKE, state=FAKE) == ps.ERR_ARG
    assert bwd(scratch=None) == ps.ERR_NULL
    big = shape(tokens=1 << 20)
    need = L.linattn_grad_scratch_bytes(big, 4, 2, 4)
    # the partial gradients of a shared head: floats for each head
    assert need >= L.linattn_grad_scratch_bytes(big, 4, 4, 4) + 2 * (1 << 20) * 4 * 64 * 4
    assert bwd(big, n=need - 300, k=rows(2), dk=rows(2)) == ps.ERR_SCRATCH
    assert bwd(shape(seqs=0), scratch=None, n=0) == ps.OK


def test_step_is_checked():
    assert step(out=rows(1)) == ps.ERR_ARG
    assert step(state=None) == ps.ERR_NULL and step(state_out=None) == ps.ERR_NULL
    assert step(slots=FAKE + 2) == ps.ERR_ALIGN and step(state=FAKE + 2) == ps.ERR_ALIGN
    assert step(pool=(1 << 36) + 1) == ps.ERR_SIZE
    assert step(shape(seqs=0), state=None, state_out=None) == ps.OK


def sample(**kw):
    base = dict(dtype=1, rows=3, vocab=1000, logits=FAKE, row_stride=1000, u=FAKE, temperature=1.0,
                top_p=1.0, min_p=0.0, top_k=0, tokens=FAKE)
    scratch, n = kw.pop("scratch", FAKE), kw.pop("n", BIG)
    base.update(kw)
    return ps.lib().sample_logits(_Sample(**base), scratch, n, None)


def test_sampling_is_checked():
    L = ps.lib()
    assert sample(dtype=3) == ps.ERR_ARG
    assert sample(vocab=(1 << 24) + 1) == ps.ERR_SIZE and sample(rows=1 << 31) == ps.ERR_SIZE
    assert sample(logits=FAKE + 1) == ps.ERR_ALIGN and sample(dtype=0, logits=FAKE + 2) == ps.ERR_ALIGN
    for name in ("u", "temperatures", "top_ks", "top_ps", "min_ps", "tokens", "logprobs", "kept"):
        assert sample(**{name: FAKE + 2}) == ps.ERR_ALIGN, name
    for name in ("logits", "u", "tokens", "scratch"):
        assert sample(**{name: None}) == ps.ERR_NULL, name
    assert sample(n=100) == ps.ERR_SCRATCH
    assert L.sample_logits(None, FAKE, BIG, None) == ps.ERR_NULL
    assert sample(rows=0, logits=None, u=None, tokens=None, scratch=None, n=0) == ps.OK
    assert L.sample_scratch_bytes(1 << 32, 10) > 0


def test_the_binding_refuses_host_tensors():
    x, g = torch.zeros(2, 5, 4, 8), torch.zeros(4)
    with pytest.raises(ValueError):
        ps.linattn(x, x, x, g)
    with pytest.raises(ValueError):
        ps.linattn_grad(x, x, x, x, g)
    with pytest.raises(ValueError):
        ps.linattn_step(x[:, 0], x[:, 0], x[:, 0], g, torch.zeros(2, 4, 8, 8))
    with pytest.raises(ValueError):
        ps.sample_logits(torch.zeros(2, 9), torch.zeros(2))
    with pytest.raises(TypeError):
        ps.linattn(x.int(), x, x, g)
    with pytest.raises(TypeError):
        ps.sample_logits([1.0], torch.zeros(1))


def test_structures_match_the_header():
    # x86-64 layout of the C structures that the binding fills
    assert ctypes.sizeof(_Rows) == 40 and ctypes.sizeof(_Shape) == 56 and ctypes.sizeof(_Sample) == 120
