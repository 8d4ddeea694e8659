"""Linear attention over every size of decay, to where its power over a chunk
or a segment is a subnormal float, or none.  Tolerances as in test_gpu_linattn."""
import numpy as np
import pytest
import torch

import prefix_scan_amd as ps
from tests import linattn_ref as ref
from tests.test_gpu_linattn import DTYPES, SCALE, host, make, near

pytestmark = pytest.mark.gpu

# e^(32 g) and e^(64 g) from a normal number to zero, closely where they are
# subnormal; e^(256 g) and further: segments.
FAST = np.concatenate([-np.linspace(1.30, 1.70, 17), -np.linspace(2.65, 3.30, 14)])
SLOW = np.concatenate([-np.linspace(0.30, 0.42, 9), -np.geomspace(1e-4, 1.0, 9), [-5.0, -20.0, -90.0, -1e4]])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", [(150, 0, 66), (700,)])
@pytest.mark.parametrize("decays", [FAST, SLOW], ids=["fast", "slow"])
def test_every_decay(decays, lens, dtype):
    heads, dk, dv = len(decays), 16, 24
    x = make(lens, heads, heads, heads, dk, dv, dtype, 110)
    x["g"] = torch.from_numpy(decays.astype(np.float32))
    names = ("do", "q", "k", "v")
    args = [x[n].cuda() for n in names]
    g, ends = x["g"].cuda(), x["ends"].cuda()
    state, dlast = x["state"].cuda(), x["dlast"].cuda()
    h = [host(x[n]) for n in names]
    a = [np.abs(t) for t in h]
    terms = max(lens) + dk + dv
    got = ps.linattn(*args[1:], g, SCALE, ends, state, want_state=True)
    want = ref.forward(*h[1:], x["g"].numpy(), SCALE, lens, host(x["state"]))
    size = ref.forward(*a[1:], x["g"].numpy(), SCALE, lens, np.abs(host(x["state"])))
    near(got[0], want[0], size[0], dtype, terms, "out")
    near(got[1], want[1], size[1], dtype, terms, "state", state=True)
    got = ps.linattn_grad(*args, g, SCALE, ends, state, dlast, True)
    want = ref.backward(*h, x["g"].numpy(), SCALE, lens, host(x["state"]), host(x["dlast"]))
    size = ref.backward(*a, x["g"].numpy(), SCALE, lens, np.abs(host(x["state"])), np.abs(host(x["dlast"])))
    for i, name in enumerate(("dq", "dk", "dv")):
        near(got[i], want[i], size[i], dtype, terms, name)
    near(got[3], want[3], size[3], dtype, terms, "dstate", state=True)
