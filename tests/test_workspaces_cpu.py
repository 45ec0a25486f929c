"""The workspaces that the binding keeps for callers that pass none (host logic: no GPU is needed)."""
import weakref

import pytest

import top_support_capture_gb300 as sfc
from top_support_capture_gb300 import speculative

torch = pytest.importorskip("torch")
DEV = torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def capture(monkeypatch):
    """A stand-in for the streams' captures: capture["id"] is the one that every stream takes part in."""
    state = {"id": 0}
    monkeypatch.setattr(sfc, "allocate_workspace", lambda n, device: torch.zeros(n, dtype=torch.uint8))
    monkeypatch.setattr(sfc, "_capture_id", lambda handle: state["id"])
    return state


def test_one_per_stream_of_a_power_of_two():
    w = sfc._Workspaces("workspace_size")
    a = w.get(1000, DEV, 7)
    assert a.numel() == 1024 and not a.any()
    assert w.get(3, DEV, 7) is a and w.get(1024, DEV, 7) is a
    assert w.get(3, DEV, 8) is not a and w.get(3, torch.device("cuda", 1), 7) is not a
    assert w.get(1025, DEV, 7).numel() == 2048


@pytest.mark.parametrize("kept", [sfc._step_workspaces, speculative._workspaces])
def test_a_captured_workspace_is_kept(kept, capture):
    """The graph may still be replayed when larger calls have come: its memory must not go to anyone else."""
    stream = 1 << 40  # no stream's handle
    kept.get(100, DEV, stream)
    capture["id"] = 1 << 50
    first = weakref.ref(kept.get(100, DEV, stream))
    capture["id"] = 0
    assert kept.get(100, DEV, stream) is not first()
    assert kept.get(5000, DEV, stream) is not first()
    assert first() is not None


def test_captures_share_with_nobody(capture):
    w = sfc._Workspaces("workspace_size")
    eager = w.get(1000, DEV, 7)
    capture["id"] = 1
    a = w.get(900, DEV, 7)
    assert a is eager and w.get(1000, DEV, 7) is a and w.get(5, DEV, 7) is a  # the calls of one capture follow each other
    capture["id"] = 2
    b = w.get(900, DEV, 7)  # no call in between
    assert b is not a and b.numel() >= 900 and w.get(100, DEV, 7) is b
    capture["id"] = 0
    again = w.get(10, DEV, 7)
    assert again is not a and again is not b and again.numel() == 1024
    capture["id"] = 3
    assert w.get(1000, DEV, 7) is again
    assert w.get(1000, DEV, 7) is again
    capture["id"] = 1
    assert w.get(1000, DEV, 7) is a


def test_a_capture_that_outgrows_its_workspace(capture):
    w = sfc._Workspaces("workspace_size")
    w.get(1000, DEV, 7), w.get(5000, DEV, 7)
    capture["id"] = 1
    w.get(5000, DEV, 7)
    capture["id"] = 2
    small = weakref.ref(w.get(10, DEV, 7))
    large = w.get(5000, DEV, 7)
    assert large.numel() >= 5000 and small() is not None and w.get(10, DEV, 7) is large


def test_a_capture_without_a_workspace_is_refused(capture):
    w = sfc._Workspaces("verify_workspace_size")
    capture["id"] = 1
    with pytest.raises(sfc.SfcError, match=r"allocate_workspace\(verify_workspace_size"):
        w.get(10, DEV, 7)
    capture["id"] = 0
    w.get(10, DEV, 7)
    capture["id"] = 2
    with pytest.raises(sfc.SfcError, match="call once before capture"):
        w.get(17, DEV, 7)
    assert w.get(16, DEV, 7).numel() == 16
