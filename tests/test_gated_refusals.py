"""Gated recurrences, embedding rows and penalties record no gradient by
themselves: tensors that ask for one are refused where one would be lost.  No
GPU: the library is a stand-in."""
import pytest
import torch

import prefix_scan_amd as ps
from tests.test_scratch_lock import library  # noqa: F401

Z = lambda *s: torch.zeros(s)  # noqa: E731
CALLS = {
    "gatescan": (ps.gatescan, lambda: dict(gate=Z(1, 4, 8), x=Z(1, 4, 8), state=Z(1, 8))),
    "gatescan_grad": (ps.gatescan_grad, lambda: dict(dout=Z(1, 4, 8), gate=Z(1, 4, 8), x=Z(1, 4, 8), out=Z(1, 4, 8),
                                                     state=Z(1, 8), dstate_out=Z(1, 8))),
    "gatescan_step": (ps.gatescan_step, lambda: dict(gate=Z(3, 8), x=Z(3, 8), state=Z(3, 8))),
    "embed_rows": (lambda weight: ps.embed_rows(weight, torch.zeros(4, dtype=torch.int64)), lambda: dict(weight=Z(5, 8))),
    "embed_grad": (lambda dout: ps.embed_grad(dout, torch.zeros(4, dtype=torch.int64), 5), lambda: dict(dout=Z(4, 8))),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_a_tensor_that_wants_a_gradient_is_refused(library, name):
    for entry in ("gatescan", "gatescan_grad", "gatescan_step", "embed_rows", "embed_grad"):
        setattr(library, entry, lambda *a: 0)
    library.gatescan_scratch_bytes = library.embed_grad_scratch_bytes = lambda *a: 512
    call, made = CALLS[name]
    call(**made())
    for which in made():
        args = made()
        args[which].requires_grad_()
        with pytest.raises(RuntimeError, match="gradient"):
            call(**args)
        with torch.no_grad():                       # as in an autograd.Function
            call(**args)


def test_penalties_are_refused_where_a_gradient_would_be_lost(library):
    library.penalize_logits = lambda *a: 0
    with pytest.raises(RuntimeError, match="gradient"):
        ps.penalize_logits(Z(2, 9).requires_grad_())
    with torch.no_grad():
        ps.penalize_logits(Z(2, 9).requires_grad_())
