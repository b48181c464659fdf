"""What the holder classes report before their first forward (no GPU needed)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402


@pytest.mark.parametrize("holder", [MM.MegaMoE, MM.MegaMoEMXFP4, H.MegaMoEHalf])
def test_no_route_was_dropped_before_the_first_forward(holder, monkeypatch):
    """megamoe_last_error reads the workspace's first word, which memory that is handed out again does not hold as 0."""
    empty = torch.empty

    def used_before(*a, **k):
        return empty(*a, **k).view(torch.uint8).fill_(0xA5).view(k.get("dtype") or torch.float32)
    monkeypatch.setattr(torch, "empty", used_before)
    moe = holder(4, 256, 8, 2, 128, device="cpu")
    assert moe.workspace[:4].view(torch.int32).item() == 0
