"""Host threads that share a stream share its scratch buffer, and a call is a
chain of kernels through it: no two calls may enqueue at once.  The library is
a stand-in here that looks whether another call is inside; no GPU is used."""
import contextlib
import threading
import time
import types

import pytest
import torch

import prefix_scan_amd as ps


class Library:
    """Answers every entry point with 0 and every size query with 64 KiB."""

    def __init__(self):
        self.inside, self.most, self.calls = {}, 0, 0
        self.guard = threading.Lock()

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 1 << 17
        if name == "libscan_scratch_init":
            return lambda *a: 0
        if name == "libscan_strerror":
            return lambda *a: b"refused"

        def call(*args):
            # the scratch buffer is the last pointer but one, before its size
            at = args[-3]
            at = at if isinstance(at, int) else at.value
            with self.guard:
                self.calls += 1
                self.inside[at] = self.inside.get(at, 0) + 1
                self.most = max(self.most, self.inside[at])
            time.sleep(0.005)
            with self.guard:
                self.inside[at] -= 1
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    stream = types.SimpleNamespace(cuda_stream=0)
    monkeypatch.setattr(ps, "lib", lambda: lib)
    monkeypatch.setattr(ps, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    for name in ("_dev_rows", "_dev_dense", "_dev_u32", "_dev_u64"):
        monkeypatch.setattr(ps, name, lambda t, *a, **k: t)
    for name in ("_scratch", "_plans"):
        monkeypatch.setattr(ps, name, {})
    return lib


X, G = torch.zeros(1, 4, 2, 8), torch.zeros(2)
I32, I64 = torch.zeros(64, dtype=torch.int32), torch.zeros(64, dtype=torch.int64)
CALLS = {
    "linattn": lambda: ps.linattn(X, X, X, G),
    "linattn_grad": lambda: ps.linattn_grad(X, X, X, X, G),
    "sample_logits": lambda: ps.sample_logits(torch.zeros(2, 9), torch.zeros(2)),
    "scan": lambda: ps.scan_exclusive_u32(I32, want_total=False),
    "scan_ex": lambda: ps.scan_u32_ex(I32, want_total=False),
    "scan_op": lambda: ps.scan_op_u32(I32, "max", want_total=False),
    "scan_op64": lambda: ps.scan_op_u64(I64, "max", want_total=False),
    "reduce_op": lambda: ps.reduce_op_u32(I32, "max", want_total=False),
    "reduce_op64": lambda: ps.reduce_op_u64(I64, "max", want_total=False),
    "runs_layout": lambda: ps.runs_layout_u32(I32, want_entries=False),
    "runs_owner": lambda: ps.runs_owner_u32(I32, I32),
    "runs_owner_all": lambda: ps.runs_owner_all_u32(I32, 64),
    "segscan": lambda: ps.segscan_u32(I32, 8),
    "segscan_flags": lambda: ps.segscan_flags_u32(I32, I32, want_nsegs=False),
    "compact": lambda: ps.compact_flags_u32(I32, want_count=False),
    "radix": lambda: ps.radix_perm_u32(I32),
    "copy": lambda: ps.copy_u32(I32, I32.clone()),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_one_call_enqueues_at_a_time(library, name):
    CALLS[name]()
    errors = []

    def work(call):
        try:
            for _ in range(3):
                call()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in (CALLS[name], CALLS[name], CALLS["sample_logits"])]
    for t in threads:
        t.start()
    for t in threads:
        t.join(20)
    assert not errors and library.calls == 10
    assert library.most == 1


def test_a_call_that_fails_lets_the_next_one_in(library, monkeypatch):
    monkeypatch.setattr(Library, "copy_u32", lambda self, *a: ps.ERR_ARG, raising=False)
    for _ in range(2):
        with pytest.raises(ps.LibscanError):
            ps.copy_u32(I32, I32.clone())
    CALLS["scan"]()
