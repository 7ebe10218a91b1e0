"""Reading the status of calls, with the device replaced by a model of it (no GPU needed)."""
import contextlib
import types

import pytest


class Devices:
    """Two devices whose current streams have handles 100 and 101; device 0 is current."""

    def __init__(self, mr, monkeypatch):
        self.current, self.asked = 0, []
        monkeypatch.setattr(mr.torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(mr.torch.cuda, "device", self.device)
        monkeypatch.setattr(mr, "_raw_stream", lambda index: 100 + index)
        monkeypatch.setattr(mr, "LIB", types.SimpleNamespace(mr_sync_status=self.sync_status))

    @contextlib.contextmanager
    def device(self, index):
        old, self.current = self.current, index
        try:
            yield
        finally:
            self.current = old

    def sync_status(self, ptr, stream):
        self.asked.append((ptr, stream, self.current))
        return 0


@pytest.mark.parametrize("index", [0, 1])
def test_status_is_read_on_the_workspaces_device(monkeypatch, index):
    from cross_model_attention_mr_b200 import mr
    d = Devices(mr, monkeypatch)
    ws = mr.Workspace.__new__(mr.Workspace)
    ws.ptr, ws.buf = 4096, types.SimpleNamespace(get_device=lambda: index)
    assert ws.sync_status() == 0
    assert d.asked == [(4096, 100 + index, index)] and d.current == 0
