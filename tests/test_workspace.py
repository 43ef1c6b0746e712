"""The PyTorch workspace: its status word, its growth (no GPU needed)."""
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
