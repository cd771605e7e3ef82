"""The routed-row operators together: a layer of microscaled FP4 experts forward and backward,
against the same steps in 64 bits with the library's roundings in their places."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M
import expert_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rel(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("act,limit", [("swiglu", 0.0), ("swiglu", 2.0), ("relu2", 0.0)])
@pytest.mark.parametrize("T,E,K,H,I,dtype", [(1, 4, 1, 64, 64, "bf16"), (37, 8, 2, 160, 96, "bf16"),
                                             (50, 6, 3, 257, 70, "f32"), (64, 16, 4, 256, 128, "f16")])
def test_layer(T, E, K, H, I, act, limit, dtype):
    dt = R.TYPES[dtype]
    g = torch.Generator().manual_seed(T + H)
    halves = 2 if act == "swiglu" else 1
    fc1 = (torch.randn(E, halves * I, H, generator=g) * H ** -0.5).to(dt)
    fc2 = (torch.randn(E, H, I, generator=g) * I ** -0.5).to(dt)
    x, dy = torch.randn(T, H, generator=g).to(dt), torch.randn(T, H, generator=g).to(dt)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :K].int()
    if T > 5:
        ids[3], ids[5, 0] = -1, -1
    w = torch.softmax(torch.randn(T, K, generator=g), 1)
    layer = M.MxExperts(fc1.to(DEV), fc2.to(DEV), act, limit)
    y, saved = layer.forward(x.to(DEV), ids.to(DEV), w.to(DEV))
    dx, dw = layer.backward(saved, dy.to(DEV))

    # the same in 64 bits, rounded where the library rounds
    q = lambda t: R.held4(t)[0]
    q1 = torch.stack([q(m) for m in fc1])
    q2 = torch.stack([q(m) for m in fc2])
    q1t = torch.stack([q(m.t()) for m in fc1])
    q2t = torch.stack([q(m.t()) for m in fc2])
    y_want, dx_want = torch.zeros(T, H).double(), torch.zeros(T, H).double()
    dw_want = torch.zeros(T, K).double()
    for t in range(T):
        for k in range(K):
            e = int(ids[t, k])
            if e < 0:
                continue
            h = (q(x[t:t + 1]) @ q1[e].t()).to(dt)
            a = R.act(h, act, limit).to(dt)
            row = (q(a) @ q2[e].t()).to(dt).double()
            y_want[t] += float(w[t, k]) * row[0]
            dw_want[t, k] = (row[0] * dy[t].double()).sum()
            drow = (float(w[t, k]) * dy[t:t + 1].double()).to(dt)
            da = (q(drow) @ q2t[e].t()).to(dt)
            dh = R.act_grad(R.kept(h, act), act, limit, da)[0].to(dt)
            dx_want[t] += (q(dh) @ q1t[e].t()).to(dt).double()[0]
    # a rounding to 16 bits that falls the other way moves a 4-bit code in a few places:
    # a step of 1/4 in one value of hundreds
    assert _rel(y, y_want) <= 2e-2 and _rel(dx, dx_want) <= 3e-2 and _rel(dw, dw_want) <= 2e-2
    if T > 5:
        assert torch.all(y[3] == 0) and torch.all(dx[3] == 0) and torch.all(dw[3] == 0)


def test_layer_in_a_graph():
    T, E, K, H, I = 200, 8, 2, 512, 256
    g = torch.Generator().manual_seed(1)
    layer = M.MxExperts((torch.randn(E, 2 * I, H, generator=g) / 22).to(DEV),
                        (torch.randn(E, H, I, generator=g) / 16).to(DEV), "swiglu")
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    dy = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :K].int().to(DEV)
    w = torch.rand(T, K, generator=g).to(DEV)

    def step():
        y, saved = layer.forward(x, ids, w)
        return (y,) + layer.backward(saved, dy)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(T, H, generator=g))
        ids.copy_(torch.rand(T, E, generator=g).argsort(1)[:, :K])
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_forward_without_a_backward_keeps_nothing():
    layer = M.MxExperts(torch.randn(4, 64, 64, device=DEV), torch.randn(4, 64, 64, device=DEV),
                        "relu2")
    x = torch.randn(5, 64, device=DEV)
    ids = torch.zeros(5, 1, dtype=torch.int32, device=DEV)
    w = torch.ones(5, 1, device=DEV)
    y, saved = layer.forward(x, ids, w, keep=False)
    again, kept = layer.forward(x, ids, w)
    assert saved.kept is None and torch.equal(y, again)
    with pytest.raises(ValueError):
        layer.backward(saved, y)
    with pytest.raises(ValueError):  # refused before the saved rows are touched
        layer.backward(kept, y.half())
    layer.backward(kept, y)
    with pytest.raises(ValueError):  # its rows hold their gradient now
        layer.backward(kept, y)
    with pytest.raises(ValueError):
        M.dispatch(layer.fc1, M.sort_routes(ids, 4))
    with pytest.raises(ValueError):
        M.MxExperts(torch.randn(4, 64, 64, device=DEV), torch.randn(4, 64, 32, device=DEV), "relu2")
