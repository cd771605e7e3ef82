"""Checkpoints that a program describes itself."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M


def test_unknown_activations_are_refused():
    codes, scales = torch.zeros(4, 1, 32, dtype=torch.uint8), torch.zeros(4, 1, 1, dtype=torch.uint8)
    with pytest.raises(ValueError):
        M.Checkpoint(codes, scales, 8, torch.float32, "gelu")
    for act in (None, "relu2"):
        assert M.Checkpoint(codes, scales, 8, torch.float32, act).act == act
