"""The routed-row calls with `stream`, from another current stream whose allocations and work
go on meanwhile: the bits of the ordinary calls."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(T, E, K, H, I, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :K].int()
    ids[torch.rand(T, K, generator=g) < 0.2] = -1
    return {"x": rnd(T, H), "h": rnd(T * K, 2 * I), "rows": rnd(T * K, H), "dout": rnd(T, H),
            "dy": rnd(T * K, I), "w": torch.rand(T, K, generator=g).to(DEV), "ids": ids.to(DEV),
            "fc": rnd(E, 40, H), "E": E}


def _calls(c, s):
    plan = M.sort_routes(c["ids"], c["E"], stream=s)
    n = plan.n_rows
    q, w = M.mx_quantize(c["x"], stream=s), M.mx_quantize(c["fc"], stream=s)
    t = M.mx_quantize_transposed(c["fc"], stream=s)
    moved = M.dispatch(q, plan, stream=s)
    kept = M.checkpoint(c["x"], stream=s)
    y, k = M.expert_act(c["h"], "swiglu", 1.5, checkpoint=True, n_rows=n, stream=s)
    live = torch.arange(c["rows"].shape[0], device=DEV)
    return {"plan": list(plan), "q": [q.codes, q.scales], "w": [w.codes, w.scales],
            "t": [t.codes, t.scales], "combine": [M.combine(c["rows"], plan, c["w"], stream=s),
                                                  M.dispatch_grad(c["rows"], plan, stream=s)],
            "kept": [kept.codes, kept.scales, M.restore(kept, stream=s)],
            "rows": [M.dispatch(c["x"], plan, stream=s), y,
                     M.expert_act_grad(k, c["dy"], n_rows=n, stream=s),
                     M.combine_grad(c["rows"], plan, c["w"], c["dout"], stream=s)[0],
                     M.mx_product(moved, w, plan.offsets, c["x"].dtype, stream=s)],
            "dw": [M.combine_grad(c["rows"], plan, c["w"], c["dout"], stream=s)[1]],
            "back": [M.mx_restore(q, stream=s)], "n": [n], "live": [live]}


def _same(got, want):
    n = int(want["n"][0])
    for name in want:
        for a, b in zip(got[name], want[name]):
            assert a.dtype == b.dtype and a.shape == b.shape, name
            if name == "rows":  # rows behind the last route are undefined
                a, b = a[:n], b[:n]
            if name in ("w", "t", "q") and a.dim() == 3:  # a row that only rounds up to even
                rows = got[name][0].shape[0]
                a, b = a[:, :rows], b[:, :rows]
            assert torch.equal(a, b), name


def _churn(seconds=0.002):
    """Work and allocations on the current stream that would meet memory given back too early."""
    torch.cuda._sleep(int(2e9 * seconds))
    for n in (1 << 8, 1 << 12, 1 << 16, 1 << 20):
        for _ in range(8):
            torch.full((n,), 255, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("T,E,K,H,I,dtype", [(9, 8, 3, 264, 96, torch.bfloat16),
                                             (700, 16, 4, 513, 130, torch.float16),
                                             (12000, 64, 3, 128, 64, torch.float32)])
def test_calls_on_a_stream(T, E, K, H, I, dtype):
    c = _inputs(T, E, K, H, I, dtype, T)
    want = _calls(c, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        _churn()
        got = _calls(c, side)
        _churn()
        side.synchronize()
        _same(got, want)
    with torch.cuda.stream(torch.cuda.Stream()):  # from a current stream of its own
        _churn()
        got = _calls(c, side)
        side.synchronize()
        _same(got, want)
    torch.cuda.synchronize()


@pytest.mark.parametrize("keep", [True, False])
def test_the_layer_on_a_stream(keep):
    T, E, K, H, I = 300, 8, 4, 520, 192
    c = _inputs(T, E, K, H, I, torch.bfloat16, 5)
    g = torch.Generator().manual_seed(6)
    fc1 = (torch.randn(E, 2 * I, H, generator=g) / 22).to(DEV)
    fc2 = (torch.randn(E, H, I, generator=g) / 14).to(DEV)

    def step(layer, s):
        y, saved = layer.forward(c["x"], c["ids"], c["w"], keep=keep, stream=s)
        return [y] + list(layer.backward(saved, c["dout"], stream=s) if keep else [])

    want = step(M.MxExperts(fc1, fc2, "swiglu", 2.0), None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer = M.MxExperts(fc1, fc2, "swiglu", 2.0, stream=side)
    for _ in range(4):
        _churn()
        got = step(layer, side)
        _churn()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()


def test_a_layer_without_tokens():
    layer = M.MxExperts(torch.randn(4, 64, 96, device=DEV), torch.randn(4, 96, 32, device=DEV),
                        "swiglu")
    x = torch.empty(0, 96, device=DEV)
    ids = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    w = torch.empty(0, 2, device=DEV)
    y, saved = layer.forward(x, ids, w)
    dx, dw = layer.backward(saved, y)
    assert y.shape == dx.shape == (0, 96) and dw.shape == (0, 2)


def test_a_layer_whose_routes_are_all_empty():
    layer = M.MxExperts(torch.randn(4, 64, 96, device=DEV), torch.randn(4, 96, 32, device=DEV),
                        "swiglu")
    x = torch.full((5, 96), float("nan"), device=DEV)
    ids = torch.full((5, 2), -1, dtype=torch.int32, device=DEV)
    y, saved = layer.forward(x, ids, torch.full((5, 2), float("nan"), device=DEV))
    dx, dw = layer.backward(saved, x)
    assert torch.all(y == 0) and torch.all(dx == 0) and torch.all(dw == 0)
