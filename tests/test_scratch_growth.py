"""A stream's scratch buffer that a larger one replaces is given back, unless
a captured graph may hold its address.  No GPU: the library is a stand-in."""
import weakref

import torch

import prefix_scan_amd as ps
from tests.test_scratch_lock import library  # noqa: F401


def grown(library, nbytes):
    with ps._scratch_at(torch.device("cpu"), 0, 0, None, nbytes) as buf:
        return buf.numel(), weakref.ref(buf)


def test_an_outgrown_buffer_is_given_back(library, monkeypatch):
    monkeypatch.setattr(ps, "_outgrown", [])
    library.libscan_scratch_captured = lambda p, n: 0
    size, first = grown(library, 1 << 18)
    assert size == 1 << 18 and first() is not None
    assert grown(library, 1 << 17)[1]() is first()            # large enough: the same
    size, second = grown(library, (1 << 18) + 1)
    assert size == 1 << 19 and first() is None and second() is not None and not ps._outgrown


def test_one_that_a_graph_may_hold_is_kept(library, monkeypatch):
    monkeypatch.setattr(ps, "_outgrown", [])
    captured = []
    library.libscan_scratch_captured = lambda p, n: int(p.value in captured)
    _, first = grown(library, 1 << 18)
    captured.append(first().data_ptr())
    _, second = grown(library, 1 << 20)
    _, third = grown(library, 1 << 22)
    assert first() is not None and second() is None and third() is not None
    assert len(ps._outgrown) == 1 and ps._outgrown[0] is first()


def test_large_buffers_grow_to_the_need(library, monkeypatch):
    monkeypatch.setattr(ps, "_outgrown", [])
    library.libscan_scratch_captured = lambda p, n: 0
    for need in (1 << 28, (1 << 28) + 4096):
        assert grown(library, need)[0] == need


def test_the_library_knows_of_no_capture_before_one():
    buf = torch.empty(4096, dtype=torch.uint8)
    assert ps.lib().libscan_scratch_captured(buf.data_ptr(), buf.numel()) == 0
    assert ps.lib().libscan_scratch_captured(None, 0) == 0
