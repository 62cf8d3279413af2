"""The cached workspaces of streams and of graphs captured on them (no GPU
needed)."""
import gc
import weakref

import pytest
import torch

import bit_weight_only_g128_gb300 as w4


@pytest.fixture
def stream(monkeypatch):
    """A stream whose capture is switched by hand, and a count of allocations."""
    state = dict(capturing=False, made=0)

    def new_workspace(nbytes, device=None):
        state["made"] += 1
        return torch.zeros(nbytes, dtype=torch.uint8)

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(w4, "new_workspace", new_workspace)
    for name, empty in (("_stream_ws", {}), ("_captured_ws", []), ("_zeroed_in_graph", set())):
        monkeypatch.setattr(w4, name, empty, raising=False)
    return state


def test_a_captured_workspace_outlives_its_replacement(stream):
    first = w4.stream_workspace(100, 0, 7)
    stream["capturing"] = True
    assert w4.stream_workspace(80, 0, 7) is first and w4.stream_workspace(100, 0, 7) is first
    stream["capturing"] = False
    alive = weakref.ref(first)
    del first
    larger = w4.stream_workspace(1000, 0, 7)
    gc.collect()
    assert alive() is not None, "replays would write to freed memory"
    assert w4.stream_workspace(100, 0, 7) is larger and stream["made"] == 2


def test_a_workspace_without_a_graph_is_freed_when_replaced(stream):
    alive = weakref.ref(w4.stream_workspace(100, 0, 7))
    w4.stream_workspace(1000, 0, 7)
    gc.collect()
    assert alive() is None


def test_a_workspace_made_in_a_capture_serves_captures_only(stream):
    """Its zero-fill is a node of the graph: before the first replay it holds anything."""
    stream["capturing"] = True
    inside = w4.stream_workspace(100, 0, 7)
    assert w4.stream_workspace(50, 0, 7) is inside
    stream["capturing"] = False
    outside = w4.stream_workspace(50, 0, 7)
    assert outside is not inside and w4.stream_workspace(50, 0, 7) is outside
    assert w4.stream_workspace(50, 0, 8) is not outside and stream["made"] == 3


def test_a_second_graph_does_not_count_on_the_firsts_zeros(stream):
    stream["capturing"] = True
    ws = w4.stream_workspace(w4.FLAG_BYTES + 100, 0, 7)  # its zero-fill: a node of the first graph
    ws[:] = 1
    assert w4.stream_workspace(100, 0, 7) is ws
    assert not ws[:w4.FLAG_BYTES].any() and ws[w4.FLAG_BYTES:].all()
    stream["capturing"] = False
    warm = w4.stream_workspace(w4.FLAG_BYTES + 100, 0, 8)
    warm[:] = 1
    stream["capturing"] = True
    assert w4.stream_workspace(100, 0, 8) is warm and warm.all()  # zeroed before: no node of its own
