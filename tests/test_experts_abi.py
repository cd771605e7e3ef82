"""The routed-row entry points without a GPU: argument checks answer before any CUDA call,
and calls without rows succeed."""
import ctypes as C

import pytest
import torch

import nvfp4_token_routed_gb300 as M

P = 4096  # a non-null, aligned pointer that nothing looks at
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from nvfp4_token_routed_gb300 import build
    build.build()
    return M.lib()


def _r(rows=4, cols=64, ld=None, data=P, dtype=0):
    return M.moe_logits(data, cols if ld is None else ld, rows, cols, dtype)


def _mx(rows=4, cols=64, codes=P, scales=P):
    return M.moe_mx(codes, scales, rows, cols)


def test_sort_checks(lib):
    def call(T=4, K=2, E=8, ids=P, i64=0, off=P, perm=P, inv=P, ws=P, n=1 << 20):
        return lib.moe_nvfp4_sort_routes(T, K, E, ids, i64, off, perm, inv, ws, n, None)

    for kw, code in ((dict(T=-1), 1), (dict(K=0), 1), (dict(E=0), 1), (dict(i64=2), 1),
                     (dict(K=33, E=64), 2), (dict(K=9), 2), (dict(E=1025), 2),
                     (dict(T=1 << 26), 2), (dict(ids=None), 1), (dict(off=None), 1),
                     (dict(perm=None), 1), (dict(inv=None), 1), (dict(T=16385, ws=None), 1),
                     (dict(ids=P + 2), 3), (dict(ids=P + 4, i64=1), 3), (dict(off=P + 1), 3),
                     (dict(perm=P + 2), 3), (dict(inv=P + 2), 3), (dict(ws=P + 16), 3),
                     (dict(n=255), 4), (dict(T=100000, n=3815), 4)):
        assert call(**kw) == code, kw
    size = M.moe_nvfp4_sort_routes_workspace_bytes
    for args in ((-1, 2, 8), (4, 0, 8), (4, 9, 8), (4, 33, 64), (4, 2, 1025), (1 << 26, 2, 8)):
        assert size(*args) == 0
    prev = 0
    for T in (0, 1, 100, 5000, 1 << 20):
        assert size(T, 8, 256) >= prev
        prev = size(T, 8, 256)
    with pytest.raises(M.MoeError):
        M.sort_routes_workspace(4, 2, 2000, device="cpu")


def test_row_checks(lib):
    def dispatch(x=None, K=2, inv=P, rows=P, ld=64):
        return lib.moe_nvfp4_dispatch(x or _r(), K, inv, rows, ld, None)

    for kw, code in ((dict(x=_r(rows=-1)), 1), (dict(x=_r(cols=0)), 1), (dict(x=_r(dtype=3)), 1),
                     (dict(x=_r(ld=63)), 1), (dict(x=_r(cols=65537)), 2), (dict(K=0), 1),
                     (dict(K=33), 2), (dict(x=_r(rows=1 << 26)), 2), (dict(ld=63), 1),
                     (dict(inv=None), 1), (dict(rows=None), 1), (dict(x=_r(data=None)), 1),
                     (dict(x=_r(data=P + 2)), 3), (dict(rows=P + 2), 3), (dict(inv=P + 2), 3)):
        assert dispatch(**kw) == code, kw
    assert dispatch(x=_r(rows=0, data=None), rows=None, inv=None) == 0
    assert lib.moe_nvfp4_dispatch(None, 2, P, P, 64, None) == 1

    def combine(rows=None, T=2, K=2, inv=P, w=P, out=P, ld=64):
        return lib.moe_nvfp4_combine(rows or _r(), T, K, inv, w, out, ld, None)

    for kw, code in ((dict(T=3), 1), (dict(T=-1), 1), (dict(K=0), 1), (dict(ld=63), 1),
                     (dict(inv=None), 1), (dict(out=None), 1), (dict(w=P + 2), 3),
                     (dict(out=P + 1, rows=_r(dtype=1)), 3)):
        assert combine(**kw) == code, kw
    assert combine(rows=_r(rows=0, data=None), T=0, inv=None, out=None) == 0

    def grad(rows=None, T=2, K=2, inv=P, w=P, dout=P, ldo=64, drows=P, ldr=64, dw=P):
        return lib.moe_nvfp4_combine_grad(rows or _r(), T, K, inv, w, dout, ldo, drows, ldr, dw,
                                          None)

    for kw, code in ((dict(T=3), 1), (dict(ldo=63), 1), (dict(ldr=63), 1), (dict(dout=None), 1),
                     (dict(drows=None), 1), (dict(rows=_r(data=None)), 1), (dict(dw=P + 2), 3),
                     (dict(dout=P + 2), 3), (dict(drows=P + 2), 3)):
        assert grad(**kw) == code, kw
    assert grad(rows=_r(rows=0, data=None), T=0) == 0


def test_checkpoint_checks(lib):
    def keep(x=None, codes=P, scales=P, n=None):
        return lib.moe_nvfp4_checkpoint(x or _r(), codes, scales, n, None)

    def back(x=None, codes=P, scales=P, n=None):
        return lib.moe_nvfp4_restore(codes, scales, x or _r(), n, None)

    for f in (keep, back):
        for kw, code in ((dict(x=_r(cols=0)), 1), (dict(x=_r(ld=63)), 1), (dict(x=_r(dtype=7)), 1),
                         (dict(x=_r(cols=(1 << 20) + 1)), 2), (dict(x=_r(rows=(1 << 26) + 1)), 2),
                         (dict(x=_r(data=None)), 1), (dict(codes=None), 1), (dict(scales=None), 1),
                         (dict(codes=P + 4), 3), (dict(n=P + 2), 3), (dict(x=_r(data=P + 2)), 3)):
            assert f(**kw) == code, kw
        assert f(x=_r(rows=0, data=None), codes=None, scales=None) == 0

    def act(h=None, a=1, L=0.0, y=P, ld=32, codes=P, scales=P, n=None):
        return lib.moe_nvfp4_expert_act(h or _r(), a, L, y, ld, codes, scales, n, None)

    for kw, code in ((dict(a=2), 1), (dict(L=-1.0), 1), (dict(L=NAN), 1), (dict(L=INF), 1),
                     (dict(a=0, L=1.0, ld=64), 1), (dict(h=_r(cols=63)), 1), (dict(ld=31), 1),
                     (dict(codes=None), 1), (dict(scales=None), 1), (dict(y=None), 1),
                     (dict(h=_r(data=None)), 1), (dict(codes=P + 4), 3), (dict(y=P + 2), 3),
                     (dict(a=0, h=_r(cols=(1 << 19) + 1), ld=1 << 20), 2)):
        assert act(**kw) == code, kw
    assert act(h=_r(rows=0, data=None), y=None, codes=None, scales=None) == 0

    def grad(dy=None, a=1, L=0.0, dh=P, ld=128, codes=P, scales=P, n=None):
        return lib.moe_nvfp4_expert_act_grad(codes, scales, a, L, dy or _r(), dh, ld, n, None)

    for kw, code in ((dict(a=-1), 1), (dict(L=NAN), 1), (dict(ld=127), 1), (dict(codes=None), 1),
                     (dict(scales=None), 1), (dict(dh=None), 1), (dict(dy=_r(data=None)), 1),
                     (dict(dy=_r(cols=(1 << 19) + 1), ld=1 << 21), 2), (dict(codes=P + 2), 3)):
        assert grad(**kw) == code, kw
    assert grad(dy=_r(rows=0, data=None), codes=None, scales=None, dh=None) == 0


def test_mx_checks(lib):
    out = (C.c_size_t * 2)()
    assert lib.moe_nvfp4_mx_sizes(3, 257, out) == 0 and list(out) == [3 * 256, 4 * 16]
    assert lib.moe_nvfp4_mx_sizes(0, 1, out) == 0 and list(out) == [0, 0]
    for rows, cols, code in ((-1, 1, 1), (1, 0, 1), (1, 65537, 2), ((1 << 26) + 1, 1, 2)):
        assert lib.moe_nvfp4_mx_sizes(rows, cols, out) == code

    def quant(x=None, q=None, n=None):
        return lib.moe_nvfp4_mx_quantize(x or _r(), q or _mx(), n, None)

    def back(x=None, q=None, n=None):
        return lib.moe_nvfp4_mx_restore(q or _mx(), x or _r(), n, None)

    for f in (quant, back):
        for kw, code in ((dict(x=_r(rows=5)), 1), (dict(x=_r(cols=32)), 1), (dict(q=_mx(codes=None)), 1),
                         (dict(q=_mx(scales=None)), 1), (dict(q=_mx(codes=P + 8)), 3),
                         (dict(q=_mx(scales=P + 8)), 3), (dict(x=_r(data=P + 2)), 3),
                         (dict(n=P + 2), 3), (dict(x=_r(data=None)), 1),
                         (dict(x=_r(cols=65537), q=_mx(cols=65537)), 2)):
            assert f(**kw) == code, kw
        assert f(x=_r(rows=0, data=None), q=_mx(0, 64, None, None)) == 0

    def trans(b=2, D=64, c=2, x=P, dt=0, q=None):
        return lib.moe_nvfp4_mx_quantize_transposed(b, D, c, x, dt, q or _mx(), None)

    for kw, code in ((dict(b=-1), 1), (dict(c=0), 1), (dict(D=0), 1), (dict(dt=3), 1),
                     (dict(c=3), 1), (dict(D=32), 1), (dict(x=None), 1), (dict(x=P + 2), 3),
                     (dict(b=1025), 2)):
        assert trans(**kw) == code, kw
    assert trans(b=0, q=_mx(rows=0), x=None) == 0

    def move(x=None, K=2, inv=P, q=None):
        return lib.moe_nvfp4_mx_dispatch(x or _mx(), K, inv, q or _mx(rows=8), None)

    for kw, code in ((dict(K=0), 1), (dict(K=33), 2), (dict(q=_mx(rows=7)), 1), (dict(inv=None), 1),
                     (dict(q=_mx(rows=8, cols=65)), 1), (dict(inv=P + 2), 3)):
        assert move(**kw) == code, kw
    assert move(x=_mx(0, 64, None, None), q=_mx(0, 64, None, None), inv=None) == 0


def test_product_checks(lib):
    def call(x=None, w=None, E=2, off=P, dt=0, out=P, ld=8):
        return lib.moe_nvfp4_mx_product(x or _mx(), w or _mx(rows=16), E, off, dt, out, ld, None)

    for kw, code in ((dict(E=0), 1), (dict(E=3), 1), (dict(off=None), 1), (dict(dt=3), 1),
                     (dict(w=_mx(rows=16, cols=65)), 1), (dict(w=_mx(0, 64)), 1), (dict(ld=7), 1),
                     (dict(out=None), 1), (dict(out=P + 2), 3), (dict(off=P + 2), 3),
                     (dict(x=_mx(codes=None)), 1), (dict(w=_mx(rows=16, scales=P + 8)), 3),
                     (dict(w=_mx(rows=2050), E=1025), 2), (dict(w=_mx(rows=65537), E=1, ld=65537), 2),
                     (dict(x=_mx(rows=1 << 26), w=_mx(rows=1 << 16), E=128, ld=512, out=P + 2), 3),
                     (dict(x=_mx(rows=1 << 26), w=_mx(rows=1 << 24), E=1024, ld=1 << 14), 2)):
        assert call(**kw) == code, kw
    assert call(x=_mx(0, 64, None, None), out=None) == 0
    assert lib.moe_nvfp4_mx_product(None, _mx(), 1, None, 0, P, 8, None) == 1
    x, w = _mx(), _mx(rows=16)
    assert lib.moe_nvfp4_selftest_product_timeout(x, w, 2, P, -1, 0, P, 8, None) == 1


def test_compiled_calls_take_no_call_that_is_not_theirs(lib):
    """They answer None, with no error left, to whatever is not an ordinary call."""
    from nvfp4_token_routed_gb300 import experts
    _calls = pytest.importorskip("nvfp4_token_routed_gb300._calls")
    assert experts._fast is _calls
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    plan = M.RoutePlan(torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), ids)
    q = M.MxTensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4, 8, dtype=torch.uint8),
                   (4, 8))
    kept = M.Checkpoint(torch.zeros(4, 1, 32, dtype=torch.uint8),
                        torch.zeros(4, 1, 1, dtype=torch.uint8), 8, x.dtype)
    odd = [x, ids, plan, q, kept, None, 3, "swiglu", (1, 2, 3), object(), x[0], x.t(), [x]]
    arity = {"sort_routes": 2, "dispatch": 3, "combine": 3, "combine_grad": 5, "checkpoint": 1,
             "restore": 1, "expert_act": 4, "expert_act_grad": 2, "mx_quantize": 1,
             "mx_raw": 3, "mx_product": 4}
    for name, n in arity.items():
        f = getattr(_calls, name)
        assert f() is None and f(*odd[:7]) is None
        for i in range(len(odd)):
            for j in range(len(odd)):
                args = [odd[i], odd[j]] + odd[2:5]
                assert f(*args[:n]) is None, (name, i, j)
    for bad in ((), (1,), ((1, 2, 3, 4), (1,) * 6, (1, 2, 3), (0,) * 11)):
        with pytest.raises(TypeError):
            _calls.attach(*bad)


def test_binding_refuses_cpu_tensors():
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    plan = M.RoutePlan(torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), ids)
    q = M.MxTensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4, 8, dtype=torch.uint8),
                   (4, 8))
    assert q.nbytes() == 4 * 128 + 32 and torch.equal(plan.n_rows, plan.offsets[3:])
    for f in (lambda: M.sort_routes(ids, 3), lambda: M.dispatch(x, plan),
              lambda: M.combine(x, plan), lambda: M.checkpoint(x), lambda: M.mx_quantize(x),
              lambda: M.expert_act(x, "relu2"), lambda: M.mx_quantize_transposed(x)):
        with pytest.raises(ValueError):
            f()
