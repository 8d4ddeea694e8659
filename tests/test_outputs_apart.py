"""Outputs whose rows share elements are refused: rows are written by different
workgroups, in no order.  Inputs may be broadcast.  No GPU: the library is a
stand-in."""
import random

import pytest
import torch

import prefix_scan_amd as ps
from tests.test_scratch_lock import library  # noqa: F401

Z = lambda *s: torch.zeros(s)  # noqa: E731
IDS = torch.zeros(4, dtype=torch.int64)

# Rows that overlap, as [B, T, D], and such that do not.
SHARED = {"all one": lambda: Z(1, 1, 8).expand(2, 4, 8), "over tokens": lambda: Z(2, 1, 8).expand(2, 4, 8),
          "over sequences": lambda: Z(1, 4, 8).expand(2, 4, 8),
          "a window": lambda: Z(100).as_strided((2, 4, 8), (40, 4, 1)),
          "sequences inside each other": lambda: Z(100).as_strided((2, 4, 8), (20, 8, 1)),
          "by one element": lambda: Z(100).as_strided((2, 4, 8), (31, 8, 1))}
APART = {"dense": lambda: Z(2, 4, 8), "turned": lambda: Z(4, 2, 8).transpose(0, 1), "spread": lambda: Z(4, 8, 20)[::2, 1::2, 3:11],
         "woven": lambda: Z(100).as_strided((2, 4, 8), (8, 16, 1)), "of one": lambda: Z(100).as_strided((2, 4, 8), (32, 8, 1))}


def calls(t):
    """What takes a [2, 4, 8] tensor as an output, and a part of it as rows of two dimensions."""
    x, rows = Z(2, 4, 8), t[:, 0]
    yield "gatescan", lambda: ps.gatescan(x, x, out=t)
    yield "gatescan packed", lambda: ps.gatescan(x[0], x[0], ends=torch.zeros(1, dtype=torch.int32), out=t[0])
    yield "dgate", lambda: ps.gatescan_grad(x, x, None, x, dgate=t)
    yield "dx", lambda: ps.gatescan_grad(x, x, None, x, dx=t)
    yield "gatescan_step", lambda: ps.gatescan_step(x[:, 0], x[:, 0], Z(2, 8), out=rows)
    yield "embed_rows", lambda: ps.embed_rows(Z(5, 8), IDS, out=t[0])
    yield "embed_grad", lambda: ps.embed_grad(Z(4, 8), IDS, 4, dweight=t[0])
    yield "penalize_logits", lambda: ps.penalize_logits(Z(4, 8), out=t[0])


def shares(t):
    at = torch.arange(t.untyped_storage().nbytes() // 4).as_strided(t.shape, t.stride(), t.storage_offset())
    return at.unique().numel() < at.numel()


@pytest.fixture
def ready(library):  # noqa: F811
    for name in ("gatescan", "gatescan_grad", "gatescan_step", "embed_rows", "embed_grad", "penalize_logits"):
        setattr(library, name, lambda *a: 0)
    return library


@pytest.mark.parametrize("which", list(SHARED))
def test_shared_rows_are_refused(ready, which):
    t = SHARED[which]()
    assert shares(t)
    refused = 0
    for name, call in calls(t):
        mine = t if name in ("gatescan", "dgate", "dx") else t[:, 0] if name == "gatescan_step" else t[0]
        if shares(mine):
            refused += 1
            with pytest.raises(ValueError, match="overlap"):
                call()
        else:
            call()
    assert refused >= 3


@pytest.mark.parametrize("which", list(APART))
def test_rows_apart_are_taken(ready, which):
    t = APART[which]()
    assert not shares(t)
    for _, call in calls(t):
        call()


def test_one_row_or_none_is_taken(ready):
    for lead in ((1, 4), (2, 0), (0, 4), (1, 1)):
        x = Z(*lead, 8)
        ps.gatescan(x, x, out=Z(1).as_strided(lead + (8,), (0, 8, 1)) if 0 in lead else Z(*lead, 8).transpose(0, 1)
                    .contiguous().transpose(0, 1))
    ps.gatescan(Z(1, 1, 8), Z(1, 1, 8), out=Z(8).as_strided((1, 1, 8), (0, 0, 1)))
    ps.embed_rows(Z(5, 8), IDS[0], out=Z(8))
    ps.embed_rows(Z(5, 8), IDS[:1], out=Z(8).expand(1, 8))


def test_heads_of_linear_attention(ready):
    ready.linattn_step = lambda *a: 0
    rows, wide = Z(2, 4, 3, 8), Z(2, 4, 9, 8)
    log_decay = Z(3)
    step = dict(log_decay=log_decay, state=Z(2, 3, 8, 8))
    ps.linattn(rows, rows, rows, log_decay, out=wide[:, :, 3:6])
    ps.linattn_grad(rows, rows, rows, rows, log_decay, dq=wide[:, :, :3], dk=wide[:, :, 3:6], dv=wide[:, :, 6:])
    ps.linattn_step(*[wide[:, 0, :3]] * 3, **step, out=wide[:, 0, 3:6])
    one = Z(2, 4, 1, 8).expand(2, 4, 3, 8)
    for call in (lambda: ps.linattn(rows, rows, rows, log_decay, out=one),
                 lambda: ps.linattn_grad(rows, rows, rows, rows, log_decay, dk=one),
                 lambda: ps.linattn_step(*[wide[:, 0, :3]] * 3, **step, out=one[:, 0])):
        with pytest.raises(ValueError, match="overlap"):
            call()


def test_broadcast_inputs_are_taken(ready):
    for shared in SHARED.values():
        t = shared()
        ps.gatescan(t, t)
        ps.gatescan_grad(t, t, t, t, blend=True)
        ps.embed_grad(t[0], IDS, 5)
        ps.penalize_logits(t[0])


def test_a_width_of_one(ready):
    x = Z(2, 4, 1)
    ps.gatescan(x, x, out=Z(8).as_strided((2, 4, 1), (1, 2, 5)))
    with pytest.raises(ValueError, match="overlap"):
        ps.gatescan(x, x, out=Z(8).as_strided((2, 4, 1), (1, 1, 1)))


def test_any_strides():
    # by the elements themselves, among them rows woven into each other
    rng, seen = random.Random(5), {True: 0, False: 0}
    for _ in range(4000):
        dims = rng.randint(1, 3)
        shape = tuple(rng.randint(1, 4) for _ in range(dims)) + (rng.randint(1, 5),)
        t = Z(400).as_strided(shape, tuple(rng.randint(0, 25) for _ in range(dims)) + (1,))
        shared = shares(t)
        seen[shared] += 1
        if shared:
            with pytest.raises(ValueError, match="overlap"):
                ps._apart(t, "out")
        else:
            ps._apart(t, "out")
    assert min(seen.values()) > 500


def test_rows_that_only_their_starts_show_apart(ready):
    # 0, 10, 20 and 15, 25, 35
    out = Z(40).as_strided((2, 3, 5), (15, 10, 1))
    assert not shares(out)
    ps.gatescan(Z(2, 3, 5), Z(2, 3, 5), out=out)
