"""Router losses, counts and the logits' gradient of large batches: the layouts of 8 and 16
lanes a row and the several rows a warp then takes, in all three types.

The 64-bit definition here is loss_refs.router over whole tensors, compared with it on a
small batch first.  Bounds as in test_gpu_router_loss.py.
"""
import pytest
import torch

import nvfp4_token_routed_gb300 as M
import loss_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 1e-5
CB, CZ = 1e-2, 1e-3
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _definition(x, ids, offsets, mask, grad, w, dw):
    """(losses, counts, tokens, dlogits, scale) as loss_refs.router."""
    T, E = x.shape
    K, S, dev = ids.shape[1], offsets.numel() - 1, x.device
    t = torch.arange(T, device=dev, dtype=offsets.dtype)
    seg = torch.searchsorted(offsets, t, right=True) - 1
    live = (seg >= 0) & (seg < S) & mask
    seg = seg.clamp(0, S - 1)
    n_s = torch.zeros(S, dtype=torch.int64, device=dev).index_add_(0, seg, live.long())
    n = int(n_s.sum())
    ok = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1).long()
    counts = torch.zeros(S * E, dtype=torch.int64, device=dev)
    counts.index_add_(0, (seg[:, None] * E + at).reshape(-1),
                      (ok & live[:, None]).long().reshape(-1))
    counts = counts.reshape(S, E)
    x = x.double()
    p, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
    f = (counts.double() * E / (K * n_s.clamp_min(1)[:, None]))[seg]
    dot = (f * p).sum(1, keepdim=True)
    on = live.double()
    losses = torch.stack([CB / n * (dot[:, 0] * on).sum(), CZ / n * (lse ** 2 * on).sum()])
    a, b = grad[0] * CB / n, (grad[1] * 2 * CZ / n * lse)[:, None]
    d = p * (a * (f - dot) + b)
    mag = p * (abs(a) * (f + dot) + b.abs())
    w, dw = w.double() * ok, dw.double()
    d.scatter_add_(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    mag.scatter_add_(1, at, w * (dw.abs() + (w * dw).abs().sum(1, keepdim=True)))
    tokens = torch.cat([n_s, n_s.sum().reshape(1)])
    return losses, counts, tokens, d * on[:, None], mag * on[:, None]


def _batch(T, E, K, S, dtype):
    g = torch.Generator(device=DEV).manual_seed(T + 1000 * E + K)
    x = torch.randn(T, E, generator=g, device=DEV) + torch.randn(E, generator=g, device=DEV)
    x = x.to(dtype)
    top = torch.topk(x.float(), K, dim=1)
    w = torch.softmax(top.values, 1)
    ids = top.indices.to(torch.int32)
    r = torch.rand(T, generator=g, device=DEV)
    ids[r < 0.1, K - 1] = -1                                # an empty slot
    if K > 1:
        again = r > 0.8
        ids[again, K // 2] = ids[again, 0]                  # an expert chosen twice
    ids[::97] = -1
    cuts = torch.randint(1, T, (S - 1,), generator=g, device=DEV).sort().values
    if S > 3:
        cuts[1] = cuts[0]                                   # a sequence without rows
    first, last = (3, T - 5) if S > 1 else (0, T)           # rows outside all sequences
    offsets = torch.cat([cuts.new_full((1,), first), cuts.clamp(first, last),
                         cuts.new_full((1,), last)]).to(torch.int32)
    mask = torch.rand(T, generator=g, device=DEV) < 0.85
    dw = torch.randn(T, K, generator=g, device=DEV) * 1e-3
    return x, ids, w, dw, offsets, mask


def test_the_definitions_agree():
    x, ids, w, dw, offsets, mask = _batch(150, 12, 4, 5, F32)
    got = _definition(x, ids, offsets, mask, (2.0, -0.5), w, dw)
    want = R.router(x.cpu(), ids.cpu(), CB, CZ, offsets.cpu(), mask.cpu(), (2.0, -0.5), w.cpu(),
                    dw.cpu())
    for a, b in zip(got, want):
        assert torch.allclose(a.cpu().double(), b.double(), rtol=1e-12, atol=1e-15)


@pytest.mark.parametrize("T,E,K,S,dtype", [
    (4096, 32, 8, 1, F32), (4096, 33, 8, 1, F32), (4097, 64, 5, 7, F32), (9729, 96, 8, 1, F32),
    (20000, 128, 1, 7, F32), (20000, 256, 16, 7, F32), (20001, 130, 9, 1, F32),
    (20000, 384, 10, 7, F32), (4096, 300, 12, 1, F32), (65536, 512, 16, 61, F32),
    (9729, 500, 8, 1, F32), (9729, 128, 32, 7, F32), (20000, 96, 12, 61, F32),
    (20000, 1000, 8, 7, F32), (40000, 200, 20, 7, F32), (40000, 333, 17, 1, F32),
    (4096, 33, 8, 1, BF16), (4096, 64, 8, 7, BF16), (20000, 96, 8, 7, BF16),
    (65536, 256, 8, 61, BF16), (9729, 250, 3, 1, BF16), (9729, 384, 16, 1, BF16),
    (20000, 512, 10, 7, BF16), (9729, 96, 32, 1, BF16), (20000, 1000, 8, 61, BF16),
    (20000, 256, 8, 61, BF16), (4099, 60, 3, 7, F16), (65536, 64, 8, 61, F16),
    (20000, 128, 4, 1, F16), (20000, 256, 8, 1, F16), (9729, 400, 12, 1, F16),
    (9729, 300, 9, 7, F16), (40000, 512, 24, 1, F16)])
def test_large_batches(T, E, K, S, dtype):
    x, ids, w, dw, offsets, mask = _batch(T, E, K, S, dtype)
    grad = (2.0, -0.5)
    kw = dict(seq_offsets=offsets, token_mask=mask)
    sc = dict(loss_grad=torch.tensor(grad, device=DEV), topk_w=w, d_topk_w=dw)
    want = _definition(x, ids, offsets, mask, grad, w, dw)
    losses, counts, tokens = M.router_loss(x, ids, CB, CZ, **kw)
    assert torch.equal(counts.long(), want[1]) and torch.equal(tokens.long(), want[2])
    assert torch.allclose(losses.double(), want[0], rtol=1e-5, atol=0.0)
    d = M.router_loss_grad(x, ids, counts, tokens, CB, CZ, **kw, **sc)
    R.check_grad(d, want[3].cpu(), want[4].cpu(), REL)
    # without the scores' part
    none = _definition(x, ids, offsets, mask, grad, w * 0, dw)
    d0 = M.router_loss_grad(x, ids, counts, tokens, CB, CZ, loss_grad=sc["loss_grad"], **kw)
    R.check_grad(d0, none[3].cpu(), none[4].cpu(), REL)
    # rows off 16-byte boundaries, 64-bit ids, the gradient in place: the same bits
    store = torch.full((T, E + 5), 77.0, dtype=dtype, device=DEV)
    view = store[:, 3:3 + E].copy_(x)
    again = M.router_loss(view, ids.long(), CB, CZ, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, (losses, counts, tokens)))
    assert torch.equal(M.router_loss_grad(view, ids.long(), counts, tokens, CB, CZ, dlogits=view,
                                          **kw, **sc), d)
    assert (store[:, :3] == 77.0).all() and (store[:, 3 + E:] == 77.0).all()
