"""Leaf logits under graph capture (no GPU needed): a living graph of the same
leaf would end the process, so the call is refused before any work."""
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import pipeline as P


def test_leaf_logits_under_capture_are_refused(monkeypatch):
    ids = torch.zeros(4, 2, dtype=torch.int32)
    leaf = torch.zeros(4, 8, requires_grad=True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="leaf logits under capture"):
        P.moe_balance_loss(leaf, ids)
    for z in (leaf * 1.0, leaf.detach()):               # these reach the library's checks
        with pytest.raises(ValueError, match="GPU"):
            P.moe_balance_loss(z, ids)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        P.moe_balance_loss(leaf, ids)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    with pytest.raises(ValueError, match="GPU"):
        P.moe_balance_loss(leaf, ids)
