"""Workspaces that the binding allocates for a call, with the allocator faked: no GPU."""
import gc

import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402


class Context:
    device = 0
    _workspace = "linear_workspace"

    def __init__(self, need):
        self._bytes = {(10, 0): need}


@pytest.fixture
def allocator(monkeypatch):
    """What the allocator was asked for, and got back; it fails above 1000 bytes."""
    log = []

    def alloc(n, stream):
        if n > 1000:
            raise torch.OutOfMemoryError("no memory")
        log.append(("alloc", n, stream))
        return 4096

    monkeypatch.setattr(osr, "_alloc", alloc)
    monkeypatch.setattr(osr, "_free", lambda p: log.append(("free", p)))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return log


def test_given_back_once(allocator):
    mem = osr._Scratch(Context(512), 10, 0, None, 7)
    assert (mem.ptr, mem.bytes) == (4096, 512)
    mem.done()
    mem.done()
    del mem
    gc.collect()
    assert allocator == [("alloc", 512, 7), ("free", 4096)]


def test_given_back_if_the_call_raises(allocator):
    mem = osr._Scratch(Context(512), 10, 0, None, 7)
    del mem
    gc.collect()
    assert allocator == [("alloc", 512, 7), ("free", 4096)]


def test_a_failed_allocation_leaves_nothing_to_give_back(allocator, monkeypatch):
    import sys
    seen = []
    monkeypatch.setattr(sys, "unraisablehook", lambda u: seen.append(u.exc_value))
    with pytest.raises(torch.OutOfMemoryError):
        osr._Scratch(Context(2000), 10, 0, None, 7)
    gc.collect()
    assert allocator == [] and seen == []


def test_none_is_needed_or_the_callers_is_used(allocator):
    assert osr._Scratch(Context(0), 10, 0, None, 7).ptr is None
    with pytest.raises(TypeError, match="workspace"):
        osr._Scratch(Context(512), 10, 0, torch.empty(512, dtype=torch.uint8), 7)
    assert allocator == []


def test_a_failed_query_leaves_nothing_to_give_back(lib, allocator, monkeypatch):
    import sys
    seen = []
    monkeypatch.setattr(sys, "unraisablehook", lambda u: seen.append(u.exc_value))
    ctx = Context(512)
    ctx.handle = None
    with pytest.raises(osr.AdamWError, match="NULL"):
        osr._Scratch(ctx, 11, 0, None, 7)
    gc.collect()
    assert allocator == [] and seen == []
