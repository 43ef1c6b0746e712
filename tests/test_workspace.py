"""The PyTorch workspace: its status word, its growth (no GPU needed)."""
import weakref

import torch


def _vx():
    import sliding_window_attention_tcgen05_b200 as vx
    return vx


def test_a_recorded_status_stays_when_the_workspace_grows():
    ws = _vx().Workspace(256, device="cpu")
    word = torch.arange(256, dtype=torch.uint8)
    ws.buf[:256] = word
    ws.get(100)
    assert ws.buf.numel() == 256 and torch.equal(ws.buf, word)
    for n in (257, 5000):
        ws.get(n)
        assert ws.buf.numel() == n and torch.equal(ws.buf[:256], word) and not ws.buf[256:].any()


def test_a_captured_buffer_outlives_the_workspaces_growth(monkeypatch):
    # A graph's replay uses the address that it was captured with.
    ws = _vx().Workspace(256, device="cpu")
    capturing = False
    monkeypatch.setattr(_vx().api, "_capturing", lambda buf: capturing)
    before = weakref.ref(ws.buf)
    ws.get(300)
    assert before() is None                       # no capture has seen it
    capturing = True
    ws.get(300)
    capturing = False
    captured = weakref.ref(ws.buf)
    for n in (400, 500):
        plain = weakref.ref(ws.buf)
        ws.get(n)
    assert captured() is not None and plain() is None
    capturing = True                              # grown inside a capture: the graph copies the old status word
    inside = weakref.ref(ws.buf)
    ws.get(600)
    capturing = False
    assert inside() is not None
    grown = weakref.ref(ws.buf)
    ws.get(700)
    assert grown() is not None
