"""Codes and scales whose tensors are given other storage, as offloading does; and copies."""
import copy
import io
import pickle

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


def _copies(t):
    with io.BytesIO() as f:
        torch.save(t, f)
        f.seek(0)
        loaded = torch.load(f, weights_only=False)
    return [copy.deepcopy(t), copy.copy(t), pickle.loads(pickle.dumps(t)), loaded]


def test_copies_describe_their_own_tensors():
    for t in (M.MxTensor(_u8(4, 128), _u8(1, 4, 8), (4, 8)),
              M.Checkpoint(_u8(4, 2, 32), _u8(4, 2, 1), 8, torch.float16, "swiglu", 2.0)):
        for other in _copies(t):
            at = other.c if type(t) is M.Checkpoint else (other.c.codes, other.c.scales)
            assert at == (other.codes.data_ptr(), other.scales.data_ptr())
            assert torch.equal(other.codes, t.codes) and torch.equal(other.scales, t.scales)
            for name in ("shape", "rows", "cols", "halves", "dtype", "act", "swiglu_limit"):
                assert getattr(other, name, None) == getattr(t, name, None)


@pytest.mark.gpu
def test_copies_have_addresses_of_their_own():
    x = torch.randn(6, 300, device="cuda")
    h = torch.randn(6, 128, device="cuda")
    y, kept = M.expert_act(h, "swiglu", 2.0, checkpoint=True)
    w = M.mx_quantize(torch.randn(2, 40, 300, device="cuda"))
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    for t, call in ((M.mx_quantize(x), lambda t: M.mx_product(t, w, off)),
                    (w, lambda t: M.mx_product(M.mx_quantize(x), t, off)),
                    (kept, lambda t: M.expert_act_grad(t, y)), (M.checkpoint(h), M.restore)):
        want = call(t)
        fresh = copy.deepcopy(t)  # of an object whose tensors nobody has asked for
        assert torch.equal(call(fresh), want)
        for other in _copies(t) + _copies(fresh):
            assert type(other) is type(t) and torch.equal(call(other), want)
            assert torch.equal(other.codes, t.codes) and torch.equal(other.scales, t.scales)
        deep = copy.deepcopy(t)
        t.codes.fill_(0)
        assert torch.equal(call(deep), want)
    layer = M.MxExperts(torch.randn(4, 64, 96, device="cuda"), torch.randn(4, 96, 64, device="cuda"),
                        "relu2")
    ids = torch.zeros(5, 1, dtype=torch.int32, device="cuda")
    args = torch.randn(5, 96, device="cuda"), ids, torch.ones(5, 1, device="cuda")
    want = layer.forward(*args)[0]
    again = copy.deepcopy(layer)
    layer.fc1.codes.fill_(0), layer.fc2.codes.fill_(0)
    del layer
    assert torch.equal(again.forward(*args)[0], want)
