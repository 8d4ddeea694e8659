"""penalize_logits records no gradient, for none of its inputs: each that asks
for one is refused where it would be lost.  No GPU: the library is a stand-in."""
import pytest
import torch

import prefix_scan_amd as ps
from tests.test_scratch_lock import library  # noqa: F401


def given():
    return dict(logits=torch.zeros(2, 9), tokens=torch.zeros((2, 3), dtype=torch.int32), repetition=torch.ones(2),
                presence=torch.zeros(2), frequency=torch.zeros(2), bias_tokens=torch.zeros((2, 4), dtype=torch.int32),
                bias_values=torch.zeros(2, 4))


@pytest.mark.parametrize("which", ["logits", "repetition", "presence", "frequency", "bias_values"])
def test_a_tensor_that_wants_a_gradient_is_refused(library, which):  # noqa: F811
    library.penalize_logits = lambda *a: 0
    ps.penalize_logits(**given())
    args = given()
    args[which].requires_grad_()
    with pytest.raises(RuntimeError, match="gradient"):
        ps.penalize_logits(**args)
    with torch.no_grad():
        assert not ps.penalize_logits(**args).requires_grad
