"""Codes and scales whose tensors are given other storage, as offloading does."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M
from nvfp4_token_routed_gb300 import experts


def _u8(*shape, device="cpu"):
    return torch.randint(1, 100, shape, dtype=torch.uint8, device=device)


def test_addresses_are_those_of_the_tensors_now():
    q = M.MxTensor(_u8(4, 128), _u8(1, 4, 8), (4, 8))
    kept = M.Checkpoint(_u8(4, 1, 32), _u8(4, 1, 1), 8, torch.float32)
    for _ in range(2):
        assert (q.c.codes, q.c.scales) == (q.codes.data_ptr(), q.scales.data_ptr())
        kept._look()
        assert kept.c == (kept.codes.data_ptr(), kept.scales.data_ptr())
        for t in (q.codes, q.scales, kept.codes, kept.scales):
            t.data = t.clone()
    q.codes.data = _u8(5, 128)
    with pytest.raises(ValueError):
        q.c
    kept.scales.untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        kept._look()


@pytest.mark.gpu
@pytest.mark.parametrize("compiled", [True, False])
def test_calls_follow_the_tensors(monkeypatch, compiled):
    M.lib()
    if not compiled:
        monkeypatch.setattr(experts, "_fast", experts._Interpreted())
    x = M.mx_quantize(torch.randn(6, 300, device="cuda"))
    w, w2 = (M.mx_quantize(torch.randn(2, 40, 300, device="cuda")) for _ in range(2))
    h = torch.randn(6, 128, device="cuda")
    y, kept = M.expert_act(h, "swiglu", checkpoint=True)
    row = M.checkpoint(h)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    calls = [lambda: M.mx_product(x, w, off), lambda: M.mx_product(x, w2, off),
             lambda: M.expert_act_grad(kept, y), lambda: M.restore(row),
             lambda: M.mx_restore(w), lambda: M.mx_restore(x)]
    want = [f() for f in calls]
    held = [x, w, kept, row]
    for t in held:
        for part in (t.codes, t.scales):  # new storage, the old one scribbled over
            old = part.data
            part.data = old.clone()
            old.fill_(77)
    assert all(torch.equal(f(), v) for f, v in zip(calls, want))
    host = [(t.codes.cpu(), t.scales.cpu()) for t in held]
    for t, (codes, scales) in zip(held, host):
        t.codes.data, t.scales.data = codes, scales
    for i in (0, 2, 3, 4, 5):
        with pytest.raises(ValueError):
            calls[i]()
    for t in held:
        t.codes.data, t.scales.data = t.codes.cuda(), t.scales.cuda()
    assert all(torch.equal(f(), v) for f, v in zip(calls, want))
    # another weight's contents under the same tensors
    w.codes.data, w.scales.data = w2.codes.clone(), w2.scales.clone()
    assert torch.equal(M.mx_product(x, w, off), want[1])
    for t in held:
        t.scales.untyped_storage().resize_(0)
    for i in (0, 2, 3, 4, 5):
        with pytest.raises(ValueError):
            calls[i]()
