"""Penalties on logits without a GPU: the C entry point refuses bad arguments
before anything is launched; the binding refuses bad tensors."""
import ctypes

import pytest
import torch

import prefix_scan_amd as ps
from prefix_scan_amd import _List, _Penalty

FAKE = 0x100000                        # never dereferenced: every case fails before launch


def call(**kw):
    base = dict(dtype=1, rows=3, vocab=1000, logits=FAKE, row_stride=1000, out=2 * FAKE, out_stride=1000,
                repetition=1.0)
    base.update(kw)
    return ps.lib().penalize_logits(_Penalty(**base), None)


def test_arguments_are_checked():
    assert ps.lib().penalize_logits(None, None) == ps.ERR_NULL
    assert call(dtype=3) == ps.ERR_ARG and call(dtype=-1) == ps.ERR_ARG
    assert call(out=FAKE, out_stride=1001) == ps.ERR_ARG
    most = 1 << 31
    for bad in (dict(vocab=(1 << 24) + 1), dict(rows=most), dict(masks=most), dict(past=_List(FAKE, 0, most, FAKE)),
                dict(bias=_List(FAKE, 0, most, FAKE))):
        assert call(**bad) == ps.ERR_SIZE, bad
    for name in ("logits", "out"):
        assert call(**{name: FAKE + 1}) == ps.ERR_ALIGN and call(**{name: None}) == ps.ERR_NULL
    for name in ("prompts", "repetitions", "presences", "frequencies", "bias_values", "mask", "mask_slots"):
        assert call(**{name: FAKE + 2}) == ps.ERR_ALIGN, name
    for name in ("past", "bias"):
        assert call(**{name: _List(FAKE + 2, 0, 1, None)}) == ps.ERR_ALIGN
        assert call(**{name: _List(FAKE, 0, 1, FAKE + 1)}) == ps.ERR_ALIGN
        assert call(**{name: _List(None, 0, 1, FAKE)}) == ps.ERR_NULL
    assert call(bias=_List(FAKE, 0, 1, None)) == ps.ERR_NULL            # values
    assert call(masks=2) == ps.ERR_NULL
    assert call(rows=0, logits=None, out=None) == ps.OK and call(vocab=0, logits=None, out=None) == ps.OK


def test_structures_match_the_header():
    assert ctypes.sizeof(_List) == 32 and ctypes.sizeof(_Penalty) == 216


def test_the_binding_refuses(monkeypatch):
    # on the host, as if it were a GPU's memory
    rows = ps._dev_rows

    def here(t, name, dtype=None, dims=None, device=None):
        try:
            return rows(t, name, dtype, dims, device)
        except ValueError as e:
            if "GPU device" not in str(e) and "must be on" not in str(e):
                raise
            return t
    monkeypatch.setattr(ps, "_dev_rows", here)
    monkeypatch.setattr(ps, "_plans", {})
    x = torch.zeros(3, 100)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bad = [
        (ValueError, dict(tokens=i(2, 5))), (ValueError, dict(tokens=i(5))), (TypeError, dict(tokens=i(3, 5).long())),
        (ValueError, dict(ends=i(3))), (ValueError, dict(tokens=i(9), ends=i(2))),
        (ValueError, dict(tokens=i(3, 3), ends=i(3))), (TypeError, dict(tokens=[1])),
        (ValueError, dict(bias_tokens=i(3, 2))), (ValueError, dict(bias_values=torch.zeros(3, 2))),
        (ValueError, dict(bias_tokens=i(3, 2), bias_values=torch.zeros(3, 1))),
        (TypeError, dict(bias_tokens=i(3, 2), bias_values=torch.zeros(3, 2).half())),
        (ValueError, dict(mask=i(3, 3))), (ValueError, dict(mask=i(2, 4))), (TypeError, dict(mask=torch.ones(3, 4).bool())),
        (ValueError, dict(mask_slots=i(3))), (ValueError, dict(mask=i(2, 4), mask_slots=i(2))),
        (TypeError, dict(repetition=torch.ones(3).half())), (ValueError, dict(presence=torch.ones(2))),
        (TypeError, dict(prompt=torch.ones(3))), (ValueError, dict(out=torch.zeros(3, 99))),
        (TypeError, dict(out=x.half())), (ValueError, dict(out=torch.zeros(1, 100).expand(3, 100))),
        (ValueError, dict(tokens=i(5, 3).t())),
    ]
    for error, kw in bad:
        with pytest.raises(error):
            ps.penalize_logits(x, **kw)
    with pytest.raises(ValueError):
        ps.penalize_logits(torch.zeros(1, (1 << 24) + 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ps.penalize_logits(torch.zeros(100))


def test_host_tensors_and_gradients_are_refused():
    with pytest.raises(ValueError):
        ps.penalize_logits(torch.zeros(2, 9))
