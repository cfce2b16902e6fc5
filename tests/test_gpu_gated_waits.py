"""Waits of the gated recurrence that run out: the call says so, whichever wait it was, and the next one runs."""
import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [40, 128, 200, 3000])
def test_a_tile_that_does_not_arrive_is_reported(cuda, monkeypatch, T, dtype):
    """LA_DEBUG_STALL=2: a block counts its tile's copies as not arrived and leaves. Of a call of one tile, and
    of a chain's last one, nobody else waits for what that block would have made known."""
    C = 72
    g = torch.Generator().manual_seed(T)
    x, ab, dy = (torch.randn(T, n, generator=g).to(dtype).to(cuda) for n in (C, 2 * C, C))
    ws = torch.empty(la.gated_scan_workspace_bytes(1, T, C, dtype), dtype=torch.uint8, device=cuda)
    saved = torch.empty(la.gated_scan_saved_bytes(1, T, C, dtype), dtype=torch.uint8, device=cuda)
    y, dx, dab = torch.empty_like(x), torch.empty_like(x), torch.empty_like(ab)

    def forward():
        la.gated_scan(None, x, ab, y, saved=saved, workspace=ws)
        return la.device_status()

    def backward():
        la.gated_scan_backward(x, ab, saved, dy, dx, dab, workspace=ws)
        return la.device_status()

    assert (forward(), backward()) == (0, 0)
    want = [v.clone() for v in (y, dx, dab)]
    keep = saved.clone()
    monkeypatch.setenv("LA_DEBUG_STALL", "2")
    assert (forward(), backward()) == (la.LA_DEV_TIMEOUT, la.LA_DEV_TIMEOUT)
    monkeypatch.delenv("LA_DEBUG_STALL")
    assert torch.equal(saved, keep)
    assert (forward(), backward()) == (0, 0)
    for u, v in zip((y, dx, dab), want):
        assert torch.equal(u, v)


@pytest.mark.parametrize("stall", ["1", "2"])
def test_blocks_that_leave_disturb_nobody(cuda, monkeypatch, stall):
    """Calls that give up early, right next to calls that do not, on two streams: shared memory that a leaving
    block has copies under way into may be another block's next. The calls that run give their own bits."""
    T, C = 3000, 256
    g = torch.Generator().manual_seed(50)
    x, ab = torch.randn(T, C, generator=g).to(cuda), torch.randn(T, 2 * C, generator=g).to(cuda)
    ws = [torch.empty(la.gated_scan_workspace_bytes(1, T, C, x.dtype), dtype=torch.uint8, device=cuda) for _ in range(2)]
    y, left = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    la.gated_scan(None, x, ab, y, workspace=ws[0])
    torch.cuda.synchronize()
    want = y.clone()
    monkeypatch.setenv("LA_WAIT_LIMIT_NS", "1000000")
    for _ in range(5):
        monkeypatch.setenv("LA_DEBUG_STALL", stall)
        la.gated_scan(None, x, ab, left, workspace=ws[1], stream=side)
        monkeypatch.delenv("LA_DEBUG_STALL")
        y.zero_()
        la.gated_scan(None, x, ab, y, workspace=ws[0])
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert la.device_status() == la.LA_DEV_TIMEOUT
