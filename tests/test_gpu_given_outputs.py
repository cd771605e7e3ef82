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


def test_a_type_that_contradicts_the_output_is_refused():
    x = torch.randn(5, 64, device=DEV)
    q, w, kept = M.mx_quantize(x), M.mx_quantize(torch.randn(7, 64, device=DEV)), M.checkpoint(x)
    out, y = torch.full((5, 64), 7.0, device=DEV), torch.full((5, 7), 7.0, device=DEV)
    for call in (lambda d: M.restore(kept, d, out=out), lambda d: M.mx_restore(q, d, out=out),
                 lambda d: M.mx_product(q, w, dtype=d, out=y)):
        for dtype in (torch.bfloat16, torch.float16, torch.float64):
            with pytest.raises(ValueError):
                call(dtype)
    assert torch.all(out == 7.0) and torch.all(y == 7.0)
    for dtype in (None, torch.float32):
        assert M.restore(kept, dtype, out=out) is out and torch.equal(out, M.restore(kept))
        assert M.mx_restore(q, dtype, out=out) is out
        assert torch.equal(out, M.mx_restore(q, torch.float32))
        assert M.mx_product(q, w, dtype=dtype, out=y) is y
        assert torch.equal(y, M.mx_product(q, w, dtype=torch.float32))
    assert M.mx_restore(q).dtype == M.mx_product(q, w).dtype == torch.bfloat16
