"""One step of the post-training example: the updates of router and head against 64-bit
gradients, the experts' rows taken one at a time through the forward."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M
import loss_refs as R
from nvfp4_token_routed_gb300 import workloads as W

pytestmark = pytest.mark.gpu


def test_one_step_updates_router_and_head_by_their_gradients():
    from nvfp4_token_routed_gb300.examples import post_training as P
    wl, dev = P.LAYER, "cuda"
    model = P.RoutedModel()
    x = W.make_x(wl, device=dev, seed=5)
    offsets = torch.tensor([0, 150, 151, wl.T], dtype=torch.int32, device=dev)
    mask = torch.arange(wl.T, device=dev) < wl.T - 20
    g = torch.Generator(device=dev).manual_seed(6)
    z, saved = model.forward(x)
    dz = (0.02 * torch.randn(z.shape, generator=g, device=dev)).to(z.dtype)
    dz[~mask] = 0
    _, r, ids, w, h = saved
    r = r.clone()
    dh = dz.double() @ model.head.double()
    codes, sf, scale = M.quantize_tokens(x)
    dw = torch.empty(wl.T, wl.K, dtype=torch.float64, device=dev)
    for k in range(wl.K):
        one = torch.zeros_like(w)
        one[:, k] = 1.0
        dw[:, k] = (M.forward(model.experts, codes, sf, scale, ids, one).double() * dh).sum(1)
    dr = R.router(r.cpu(), ids.cpu(), P.BALANCE, P.Z, offsets.cpu(), mask.cpu(), (1.0, 1.0),
                  w.cpu(), dw.cpu())[3]
    router, head = model.router.clone(), model.head.clone()
    model.step(saved, dz, offsets, mask, rate=1.0)
    # fp32 products of up to 2000 terms, whose errors add up at random: far below 1e-4
    for got, want in ((router - model.router, dr.t() @ x.cpu().double()),
                      (head - model.head, (dz.double().t() @ h.double()).cpu())):
        got = got.cpu().double()
        assert float(want.norm()) > 0.01
        assert float((got - want).norm()) <= 1e-4 * float(want.norm())
