"""The experts' activation and its gradient at the ends of the types' ranges: exact zeros,
infinities of the right sign."""
import math

import pytest
import torch

import nvfp4_token_routed_gb300 as M
import expert_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("limit", [0.0, 2.0])
def test_the_lowest_gate_gives_zero(dtype, limit):
    """s(g) is 0 there (e^-g passes fp32), so y = g 0 u and both gradients are 0.  f16's lowest,
    -65504, is far enough below -104 too."""
    low = torch.finfo(R.TYPES[dtype]).min
    h = torch.full((3, 128), low, dtype=R.TYPES[dtype], device=DEV)
    h[:, 64:96] = 1.0  # and a finite up beside the lowest one
    y, kept = M.expert_act(h, "swiglu", limit, checkpoint=True)
    assert torch.equal(y, torch.zeros_like(y))
    assert torch.equal(M.expert_act(h, "swiglu", limit), torch.zeros_like(y))
    dh = M.expert_act_grad(kept, torch.ones_like(y))
    assert torch.equal(dh, torch.zeros_like(dh))
    y, kept = M.expert_act(h, "relu2", checkpoint=True)
    want = torch.zeros_like(h)
    want[:, 64:96] = 1.0
    assert torch.equal(y, want)
    assert torch.equal(M.expert_act_grad(kept, torch.ones_like(y)), 2.0 * want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act,limit", [("swiglu", 0.0), ("relu2", 0.0)])
def test_results_past_the_type_are_infinite(act, limit, dtype):
    dt = R.TYPES[dtype]
    g = torch.Generator().manual_seed(2)
    top = math.sqrt(torch.finfo(dt).max)
    # magnitudes from an eighth of the root of the type's largest to eight times it
    h = torch.randn(40, 192, generator=g).sign() * torch.exp2(torch.rand(40, 192, generator=g) * 6 - 3)
    h = (h * top).to(dt)
    dy = torch.randn(40, 96 if act == "swiglu" else 192, generator=g).to(dt)
    dy = (dy.double() * top).to(dt)
    y, kept = M.expert_act(h.to(DEV), act, limit, checkpoint=True)
    dh = M.expert_act_grad(kept, dy.to(DEV))
    hd = R.kept(h, act)
    want_y, (want_d, weight) = R.act(h, act, limit), R.act_grad(hd, act, limit, dy)
    for got, want, rel in ((y, want_y, (8 + 1.2 * h.double().abs()[:, :want_y.shape[1]]) * 2.0 ** -23),
                           (dh, want_d, None)):
        got = got.cpu().double()
        # products in fp32 order: the last one is the first to pass fp32's range
        err = rel * want.abs() if rel is not None else 2.0 ** -23 * weight
        err = torch.minimum(err, 2.0 ** -10 * want.abs())
        far = want.abs() > 1.01 * torch.finfo(dt).max
        near = want.abs() < 0.99 * torch.finfo(dt).max
        assert far.any() and near.any()
        assert torch.equal(got[far], torch.sign(want[far]) * math.inf)
        tol = R.half_step(dt) * want.abs() + err + R.tiny(dt)
        assert torch.all(((got - want).abs() <= tol)[near])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act,limit", [("swiglu", 0.0), ("swiglu", 2.0), ("relu2", 0.0)])
def test_the_largest_gradients_where_the_slope_is_zero(act, limit, dtype):
    """Factors whose product passes fp32 come to a result of 0 where the slope is 0."""
    dt = R.TYPES[dtype]
    top = torch.finfo(dt).max
    h = torch.full((2, 128), 0.9 * top, dtype=dt)
    h[:, :64] = -0.9 * top  # (relu2 has no halves: its first 64 values)
    dy = torch.tensor([[top], [-top]], dtype=dt).expand(2, 64 if act == "swiglu" else 128).contiguous()
    _, kept = M.expert_act(h.to(DEV), act, limit, checkpoint=True)
    dh = M.expert_act_grad(kept, dy.to(DEV))
    assert torch.equal(dh[:, :64], torch.zeros_like(dh[:, :64]))
    want = R.act_grad(R.kept(h, act), act, limit, dy)[0].to(dt)
    assert torch.equal(dh.cpu(), want)
