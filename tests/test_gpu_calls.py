"""The compiled calls of the binding against the interpreted ones: the same results, the same
errors, no reference kept or lost."""
import gc
import sys

import pytest
import torch

import nvfp4_token_routed_gb300 as M
from nvfp4_token_routed_gb300 import experts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def compiled():
    M.lib()
    calls = pytest.importorskip("nvfp4_token_routed_gb300._calls")
    assert experts._fast is calls
    return calls


def _case(seed, T=50, E=8, K=3, H=264, I=96, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)
    return {"x": rnd(T, H + 5)[:, 2:2 + H] if seed % 2 else rnd(T, H), "h": rnd(T * K, 2 * I),
            "rows": rnd(T * K, H), "dout": rnd(T, H), "dy": rnd(T * K, I),
            "w": torch.rand(T, K, generator=g).to(DEV), "fc": rnd(E, 40, H), "one": rnd(33, H),
            "ids": torch.rand(T, E, generator=g).argsort(1)[:, :K].to(
                torch.int64 if seed % 2 else torch.int32).to(DEV), "E": E}


def _all(c):
    plan = M.sort_routes(c["ids"], c["E"])
    rows = M.dispatch(c["x"], plan)
    given = torch.zeros(rows.shape[0], rows.shape[1] + 3, dtype=rows.dtype, device=DEV)[:, 1:-2]
    M.dispatch(c["x"], plan, rows=given)
    out = [*plan, rows, given, M.combine(rows, plan, c["w"]), M.combine(rows, plan),
           M.dispatch_grad(c["rows"], plan), *M.combine_grad(c["rows"], plan, c["w"], c["dout"]),
           *M.combine_grad(c["rows"], plan, None, c["dout"], drows=given)]
    kept = M.checkpoint(c["x"])
    out += [kept.codes, kept.scales, M.restore(kept)]
    for act, limit in (("swiglu", 0.0), ("swiglu", 1), ("relu2", 0.0)):
        dy = c["dy"] if act == "swiglu" else c["h"]
        y, k = M.expert_act(c["h"], act, limit, checkpoint=True)
        out += [y, M.expert_act(c["h"], act, limit), k.codes, k.scales, M.expert_act_grad(k, dy)]
    q = M.mx_quantize(rows)
    w, one = M.mx_quantize(c["fc"]), M.mx_quantize(c["one"])
    stack = M.MxTensor(w.codes, w.scales, list(w.shape))
    out += [q.codes, q.scales, w.codes, w.scales]
    out += [M.mx_product(q, w, plan.offsets, torch.float32), M.mx_product(q, w, plan.offsets),
            M.mx_product(q, stack, plan.offsets), M.mx_product(q, one), M.mx_product(M.MxTensor(q.codes, q.scales, q.shape), one),
            M.restore(M.Checkpoint(kept.codes, kept.scales, kept.cols, kept.dtype))]
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("seed", [0, 1])
def test_the_same_results(compiled, monkeypatch, seed, dtype):
    c = _case(seed, dtype=dtype)
    fast = _all(c)
    monkeypatch.setattr(experts, "_fast", experts._Interpreted())
    slow = _all(c)
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
        assert torch.equal(a, b)


def test_without_the_short_allocation(compiled, monkeypatch):
    """Both ways allocate by torch.empty_strided where torch lacks its shorter form."""
    c = _case(1)
    want = _all(c)
    with monkeypatch.context() as m:
        m.setattr(experts, "_empty", experts._empty_by_torch)
        experts._attach(M.lib())
        fast = _all(c)
        m.setattr(experts, "_fast", experts._Interpreted())
        slow = _all(c)
    experts._attach(M.lib())
    assert experts._fast is compiled
    for a, b, d in zip(want, fast, slow):
        assert torch.equal(a, b) and torch.equal(a, d)
        assert a.stride() == b.stride() == d.stride()


def test_the_same_attributes(compiled, monkeypatch):
    c = _case(0)

    def about():
        k1, (_, k2) = M.checkpoint(c["x"]), M.expert_act(c["h"], "swiglu", 2, checkpoint=True)
        q = M.mx_quantize(c["x"])
        return [[type(k), k.rows, k.halves, k.cols, k.dtype, k.act, k.swiglu_limit, k.device,
                 k.nbytes()] for k in (k1, k2)] + [[type(q), q.shape, q.device, q.nbytes(),
                                                    q.c.rows, q.c.cols]]

    fast = about()
    monkeypatch.setattr(experts, "_fast", experts._Interpreted())
    assert fast == about()


def test_ordinary_calls_are_compiled(compiled):
    c = _case(0)
    plan = compiled.sort_routes(c["ids"], c["E"])
    assert type(plan) is M.RoutePlan
    for r in (compiled.dispatch(c["x"], plan, None), compiled.combine(c["rows"], plan, c["w"]),
              compiled.combine_grad(c["rows"], plan, c["w"], c["dout"], None),
              compiled.checkpoint(c["x"]), compiled.restore(compiled.checkpoint(c["x"])),
              compiled.expert_act(c["h"], "swiglu", 0.0, True),
              compiled.expert_act_grad(compiled.expert_act(c["h"], "swiglu", 0.0, True)[1], c["dy"]),
              compiled.mx_quantize(c["x"]),
              compiled.mx_product(compiled.mx_quantize(c["x"]), M.mx_quantize(c["one"]), None,
                                  torch.float16)):
        assert r is not None


@pytest.mark.parametrize("T,K", [(16384, 2), (16385, 2), (40000, 3)])
def test_sorts_with_a_workspace(compiled, monkeypatch, T, K):
    ids = torch.randint(-2, 70, (T, K), generator=torch.Generator().manual_seed(T)).to(DEV)
    fast = [compiled.sort_routes(ids, 64), compiled.sort_routes(ids.int(), 64)]
    monkeypatch.setattr(experts, "_fast", experts._Interpreted())
    for got in fast:
        for a, b in zip(got, M.sort_routes(ids, 64)):
            assert a.shape == b.shape and torch.equal(a, b)


def test_other_calls_are_not(compiled):
    c = _case(0)
    plan = M.sort_routes(c["ids"], c["E"])
    q, w = M.mx_quantize(c["x"]), M.mx_quantize(c["fc"])
    _, k = M.expert_act(c["h"], "swiglu", checkpoint=True)
    bad = torch.zeros(c["E"] + 1, device=DEV)
    for f, args in ((compiled.sort_routes, (c["ids"].float(), 8)), (compiled.sort_routes, (c["ids"], 2)),
                    (compiled.sort_routes, (c["ids"].t(), 64)), (compiled.sort_routes, (c["ids"][:0], 8)),
                    (compiled.dispatch, (c["x"][:4], plan, None)), (compiled.dispatch, (q, plan, None)),
                    (compiled.dispatch, (c["x"], plan, c["rows"][:, :40])),
                    (compiled.dispatch, (c["x"], tuple(plan), None)),
                    (compiled.combine, (c["x"], plan, None)),
                    (compiled.combine, (c["rows"], plan, c["w"].half())),
                    (compiled.combine, (c["rows"], plan, c["w"].t())),
                    (compiled.combine_grad, (c["rows"], plan, None, c["dout"].float(), None)),
                    (compiled.checkpoint, (c["x"].double(),)), (compiled.checkpoint, (c["x"].t(),)),
                    (compiled.restore, (k,)), (compiled.restore, (q,)),
                    (compiled.expert_act, (c["h"], "gelu", 0.0, True)),
                    (compiled.expert_act, (c["h"], "relu2", 1.0, True)),
                    (compiled.expert_act, (c["h"], "swiglu", float("nan"), True)),
                    (compiled.expert_act, (c["h"], "swiglu", "1", True)),
                    (compiled.expert_act_grad, (k, c["h"])),
                    (compiled.expert_act_grad, (M.checkpoint(c["x"]), c["x"])),
                    (compiled.mx_quantize, (c["fc"],)), (compiled.mx_product, (q, w, None, q)),
                    (compiled.mx_raw, (w.codes, w.scales, (8, 41, 264))),
                    (compiled.mx_raw, (w.codes, w.scales, [8, 40, 264])),
                    (compiled.mx_raw, (w.codes, w.scales, (0, 40, 264))),
                    (compiled.mx_raw, (w.codes, w.scales, (8, 8, 5, 264))),
                    (compiled.mx_raw, (w.codes, w.scales, (2 ** 40, 40, 264))),
                    (compiled.mx_raw, (w.codes[:, ::2], w.scales, (8, 40, 264))),
                    (compiled.mx_raw, (w.codes.cpu(), w.scales, w.shape)),
                    (compiled.mx_raw, (w.scales, w.codes, w.shape)),
                    (compiled.mx_product, (q, w, None, torch.float32)),
                    (compiled.mx_product, (q, w, bad, torch.float32)),
                    (compiled.mx_product, (w, w, plan.offsets, torch.float32)),
                    (compiled.mx_product, (q, w, plan.offsets, torch.float64))):
        assert f(*args) is None, (f, args)


def test_references_and_memory(compiled):
    c = _case(1)
    plan = M.sort_routes(c["ids"], c["E"])
    q, w = M.mx_quantize(c["x"]), M.mx_quantize(c["one"])
    _, k = M.expert_act(c["h"], "swiglu", checkpoint=True)
    watched = [c["x"], c["rows"], c["w"], c["dout"], c["h"], c["ids"], *plan, plan, q, w, k,
               q.shape, k.c, torch.bfloat16, torch.uint8, M.MxTensor, M.Checkpoint, M.RoutePlan,
               experts._empty]

    def some(n):
        for _ in range(n):
            _all(c)
            M.mx_product(q, w)
            M.expert_act_grad(k, c["dy"])
            compiled.mx_product(q, w, None, torch.float64)
            compiled.combine_grad(c["rows"], plan, c["w"].half(), c["dout"], None)
            compiled.expert_act(c["h"], "swiglu", float("nan"), True)
        torch.cuda.synchronize()
        gc.collect()

    some(3)
    counts, used = [sys.getrefcount(o) for o in watched], torch.cuda.memory_allocated()
    some(50)
    after = [sys.getrefcount(o) for o in watched]
    assert torch.cuda.memory_allocated() == used
    assert all(abs(a - b) <= 2 for a, b in zip(after, counts)), (counts, after)
    # results outlive what they were made from
    kept = M.checkpoint(c["x"].clone())
    r = M.restore(kept)
    codes = kept.codes
    del kept
    junk = [torch.full((1 << 16,), 9, dtype=torch.uint8, device=DEV) for _ in range(8)]
    assert torch.equal(codes, M.checkpoint(c["x"]).codes) and torch.equal(r, M.restore(
        M.checkpoint(c["x"])))
    del junk


def test_current_stream(compiled):
    """New results belong to the current stream, and so does the work."""
    x = torch.randn(2000, 1024, device=DEV)
    want = M.restore(M.checkpoint(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = M.restore(M.checkpoint(x))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = M.restore(M.checkpoint(x))
    x.mul_(2.0)
    graph.replay()
    assert torch.equal(got, M.restore(M.checkpoint(x)))
