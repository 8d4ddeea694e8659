"""Embedding rows of batches without tokens, whichever of their dimensions is
empty.  No GPU: the library is a stand-in."""
import pytest
import torch

import prefix_scan_amd as ps
from tests.test_scratch_lock import library  # noqa: F401

EMPTY = [(0,), (3, 0), (0, 3), (2, 0, 4), (0, 2, 4), (2, 4, 0), (0, 0)]


@pytest.mark.parametrize("lead", EMPTY)
def test_no_rows_are_evenly_spaced(lead):
    for t in (torch.zeros(lead + (8,)), torch.zeros(lead + (16,))[..., 3:11]):
        assert ps._spaced(t, "x") >= 0


@pytest.mark.parametrize("lead", EMPTY)
def test_lookups_and_gradients_of_no_tokens(library, lead):
    seen = []
    library.embed_rows = lambda shape, *a: seen.append(("rows", shape.tokens)) or 0
    library.embed_grad = lambda shape, *a: seen.append(("grad", shape.tokens)) or 0
    ids, rows = torch.zeros(lead, dtype=torch.int64), torch.zeros(lead + (8,))
    assert ps.embed_rows(torch.zeros(5, 8), ids).shape == rows.shape
    assert ps.embed_rows(torch.zeros(5, 8), ids, out=rows) is rows
    assert ps.embed_grad(rows, ids, 5).shape == (5, 8)
    held = torch.ones(5, 8)
    assert ps.embed_grad(rows, ids, 5, dweight=held, accumulate=True) is held
    assert seen == [("rows", 0), ("rows", 0), ("grad", 0), ("grad", 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("lead", EMPTY)
def test_on_the_gpu(lead):
    ids = torch.zeros(lead, dtype=torch.int64, device="cuda")
    weight, rows = torch.ones(1000, 24, device="cuda"), torch.zeros(lead + (24,), device="cuda")
    assert ps.embed_rows(weight, ids, out=rows) is rows
    held = torch.ones(1000, 24, device="cuda")
    assert bool((ps.embed_grad(rows, ids, 1000, dweight=held, accumulate=True) == 1).all())
    assert not ps.embed_grad(rows, ids, 1000, dweight=held).any()
    assert not ps.embed_grad(rows, ids, 1000).any()
