"""The gated recurrence's definition in 64 bits: its gradient against
differences.  No GPU."""
import numpy as np
import pytest

from tests import gatescan_ref as ref


@pytest.mark.parametrize("blend", [False, True])
@pytest.mark.parametrize("form", ["decay", "log", "sigmoid"])
def test_the_gradient_is_that_of_differences(form, blend):
    rng = np.random.default_rng(3)
    lens, d = [3, 0, 1, 5], 2
    n = sum(lens)
    gate = {"decay": rng.uniform(-0.9, 0.9, (n, d)), "log": -rng.exponential(0.5, (n, d)),
            "sigmoid": rng.normal(1, 2, (n, d))}[form]
    x, state = rng.normal(size=(n, d)), rng.normal(size=(4, d))
    dout, dlast = rng.normal(size=(n, d)), rng.normal(size=(4, d))

    def total(gate, x, state):
        a, rest = ref.gates(gate, form)
        out, last = ref.forward(a, rest * x if blend else x, lens, state)
        return (out * dout).sum() + (last * dlast).sum()

    a, rest = ref.gates(gate, form)
    out, _ = ref.forward(a, rest * x if blend else x, lens, state)
    dh, dstate = ref.backward(dout, a, lens, dlast)
    prev = ref.before(out, lens, state)
    grads = (dh * (prev - x if blend else prev) * ref.slope(a, rest, form), dh * rest if blend else dh, dstate)
    step = 1e-6
    for i, given in enumerate((gate, x, state)):
        for at in np.ndindex(given.shape):
            args = [t.copy() for t in (gate, x, state)]
            args[i][at] += step
            up = total(*args)
            args[i][at] -= 2 * step
            # second differences of order 1, so step^2, and rounding over step
            assert abs((up - total(*args)) / (2 * step) - grads[i][at]) < 1e-7


def test_gates():
    a, rest = ref.gates([-800.0, -1.0, 0.0, 2.0, 800.0], "sigmoid")
    assert np.allclose(a + rest, 1) and a[0] == 0 and rest[4] == 0 and a[2] == 0.5
