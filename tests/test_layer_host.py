"""Host-side behaviour of the Python binding around the cache operators (no GPU, no launch)."""

import weakref

import pytest
import torch

from token_level_sparse_fp8_b200 import api


@pytest.fixture
def cpu_workspace(monkeypatch):
    """A workspace over host memory whose calls into the library do nothing."""
    state = {"capturing": False}
    monkeypatch.setattr(api, "call", lambda *a: None)
    monkeypatch.setattr(api, "_stream", lambda device: 0)
    monkeypatch.setattr(api, "_capturing", lambda: state["capturing"], raising=False)
    return api.Workspace("cpu"), state


def test_workspace_keeps_what_a_captured_graph_holds(cpu_workspace):
    ws, state = cpu_workspace
    state["capturing"] = True
    ws.get(1000)
    held = weakref.ref(ws.buf)
    ws.get(500)
    state["capturing"] = False
    ws.get(5000)  # replaces the buffer
    assert held() is not None and ws.buf.numel() == 5000
    dropped = weakref.ref(ws.buf)
    ws.get(9000)
    assert dropped() is None  # no graph was given that one
    assert held() is not None
