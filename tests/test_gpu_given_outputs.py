"""Outputs that the caller gives: written and returned themselves, of their own type."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_restored_stacks():
    w = M.mx_quantize(torch.randn(3, 40, 70, device=DEV))
    want = M.mx_restore(w, torch.float32)
    assert want.shape == (3, 40, 70)
    out = torch.empty(120, 70, device=DEV)
    assert M.mx_restore(w, out=out) is out and torch.equal(out.view(3, 40, 70), want)
    wide = torch.empty(120, 80, device=DEV)[:, 3:73]
    assert M.mx_restore(w, out=wide) is wide and torch.equal(wide, out)
