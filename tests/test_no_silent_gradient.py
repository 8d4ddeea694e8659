"""Linear attention records no gradient by itself: tensors that ask for one
are refused where one would be recorded.  No GPU: the library is a stand-in."""
import pytest
import torch

import prefix_scan_amd as ps
from tests.test_scratch_lock import library  # noqa: F401

Z = lambda *s: torch.zeros(s)  # noqa: E731
CALLS = {
    "linattn": (ps.linattn, lambda: dict(q=Z(1, 4, 2, 8), k=Z(1, 4, 2, 8), v=Z(1, 4, 2, 8), log_decay=Z(2),
                                         state=Z(1, 2, 8, 8))),
    "linattn_grad": (ps.linattn_grad, lambda: dict(dout=Z(1, 4, 2, 8), q=Z(1, 4, 2, 8), k=Z(1, 4, 2, 8),
                                                   v=Z(1, 4, 2, 8), log_decay=Z(2), state=Z(1, 2, 8, 8),
                                                   dstate_out=Z(1, 2, 8, 8))),
    "linattn_step": (ps.linattn_step, lambda: dict(q=Z(3, 2, 8), k=Z(3, 2, 8), v=Z(3, 2, 8), log_decay=Z(2),
                                                   state=Z(3, 2, 8, 8))),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_a_tensor_that_wants_a_gradient_is_refused(library, name):
    library.linattn_step = lambda *a: 0             # it has no scratch to look at
    call, made = CALLS[name]
    call(**made())
    for which in made():
        args = made()
        args[which].requires_grad_()
        with pytest.raises(RuntimeError, match="gradient"):
            call(**args)
        with torch.no_grad():                       # as in an autograd.Function
            call(**args)


def test_sampling_takes_them(library):
    # tokens have no gradient to lose
    tokens = ps.sample_logits(Z(2, 9).requires_grad_(), Z(2))[0]
    assert not tokens.requires_grad


def test_an_autograd_function_gets_through(library):
    class F(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, g):
            ctx.save_for_backward(q, k, v, g)
            return ps.linattn(q, k, v, g)[0]

        @staticmethod
        def backward(ctx, dout):
            return (*ps.linattn_grad(dout.contiguous(), *ctx.saved_tensors)[:3], None)

    rows = [Z(1, 4, 2, 8).requires_grad_() for _ in range(3)]
    F.apply(*rows, Z(2)).sum().backward()
    assert all(t.grad is not None for t in rows)
