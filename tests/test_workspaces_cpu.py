"""The workspaces that the binding keeps for callers that pass none (host logic: no GPU is needed)."""
import weakref

import pytest

import top_support_capture_gb300 as sfc
from top_support_capture_gb300 import speculative

torch = pytest.importorskip("torch")
DEV = torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def _host_memory(monkeypatch):
    monkeypatch.setattr(sfc, "allocate_workspace", lambda n, device: torch.zeros(n, dtype=torch.uint8))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def test_one_per_stream_of_a_power_of_two():
    w = sfc._Workspaces("workspace_size")
    a = w.get(1000, DEV, 7)
    assert a.numel() == 1024 and not a.any()
    assert w.get(3, DEV, 7) is a and w.get(1024, DEV, 7) is a
    assert w.get(3, DEV, 8) is not a and w.get(3, torch.device("cuda", 1), 7) is not a


@pytest.mark.parametrize("kept", [sfc._step_workspaces, speculative._workspaces])
def test_a_replaced_workspace_is_kept(kept):
    """A graph captured with it may still be replayed: its memory must not go to anyone else."""
    stream = 1 << 40  # no stream's handle
    first = weakref.ref(kept.get(100, DEV, stream))
    assert kept.get(5000, DEV, stream) is not first()
    assert first() is not None


def test_a_capture_without_a_workspace_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(sfc.SfcError, match=r"allocate_workspace\(verify_workspace_size"):
        sfc._Workspaces("verify_workspace_size").get(10, DEV, 7)
