"""Routes sorted by expert, token rows to their routes' rows and back, and the gradients,
against plain definitions in 64 bits.

Bounds: a copy is exact.  combine adds at most K terms in fp32 (each product and sum half of
2^-23 of what it holds) and rounds once; combine's gradient rounds one fp32 product; a dot
product of H terms passes at most H / 32 + 64 additions in a chain (a lane's own terms, the
warp's, the segments', the warps').
"""
import pytest
import torch

import nvfp4_token_routed_gb300 as M
import expert_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ids(T, E, K, empty, seed, dtype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :K].to(dtype)
    return torch.where(torch.rand(T, K, generator=g) < empty, -1, ids).contiguous()


def _check_plan(plan, ids, E):
    # whole-tensor definition: stable order of the keys
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    n = int((key < E).sum())
    offsets = torch.searchsorted(key[order].contiguous(), torch.arange(E + 1))
    assert torch.equal(plan.offsets.cpu().long(), offsets)
    want = torch.where(torch.arange(flat.numel()) < n, order, -1)
    assert torch.equal(plan.perm.cpu().long(), want)
    inv = torch.full((flat.numel(),), -1)
    inv[order[:n]] = torch.arange(n)
    assert torch.equal(plan.inv.cpu().long().reshape(-1), inv)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 1024, 32), (5, 8, 8), (33, 60, 4), (512, 256, 8),
                                   (513, 256, 8), (128, 1000, 32), (4097, 1, 1), (4096, 384, 6),
                                   (5000, 1024, 3), (20000, 33, 10), (4096, 8, 8),
                                   (4097, 8, 8), (128, 8, 8), (129, 1024, 8), (1025, 7, 1), (32768, 64, 1), (32767, 40, 1), (32769, 2, 1)])
@pytest.mark.parametrize("empty", [0.0, 0.3])
def test_sort(T, E, K, empty):
    for dtype in (torch.int32, torch.int64):
        ids = _ids(T, E, K, empty, T + K, dtype)
        _check_plan(M.sort_routes(ids.to(DEV), E), ids, E)


def test_definitions_agree():
    ids = _ids(40, 7, 3, 0.3, 1)
    offsets, perm, inv = R.sort(ids, 7)
    plan = M.sort_routes(ids.to(DEV), 7)
    assert torch.equal(plan.offsets.cpu(), offsets) and torch.equal(plan.perm.cpu(), perm)
    assert torch.equal(plan.inv.cpu(), inv)


@pytest.mark.parametrize("T", [7, 3000, 9000])
def test_sort_bad_repeated_and_missing_ids(T):
    E, K = 16, 4
    ids = torch.randint(0, E, (T, K), generator=torch.Generator().manual_seed(2))  # repeats
    ids[T // 2] = -1
    ws = M.sort_routes_workspace(T, K, E)
    ws.fill_(0xA5)
    _check_plan(M.sort_routes(ids.to(DEV), E, ws=ws), ids, E)
    assert M.moe_nvfp4_read_status(ws) == 0
    for bad in (E, -2, 1 << 40, -(1 << 40), (1 << 32) + 3):
        worse = ids.clone()
        worse[T - 1, 1] = bad
        _check_plan(M.sort_routes(worse.to(DEV), E, ws=ws), worse, E)
        assert M.moe_nvfp4_read_status(ws) == 7
    all_empty = torch.full((T, K), -1, dtype=torch.int32)
    plan = M.sort_routes(all_empty.to(DEV), E, ws=ws)
    _check_plan(plan, all_empty, E)
    assert M.moe_nvfp4_read_status(ws) == 0 and int(plan.n_rows) == 0


def test_sort_large():
    ids = torch.randint(0, 256, (1 << 19, 8), dtype=torch.int32,
                        generator=torch.Generator().manual_seed(4))
    _check_plan(M.sort_routes(ids.to(DEV), 256), ids, 256)


def test_no_tokens():
    ids = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    plan = M.sort_routes(ids, 8)
    assert plan.offsets.tolist() == [0] * 9 and plan.perm.numel() == 0
    x = torch.empty(0, 64, device=DEV)
    assert M.dispatch(x, plan).shape == (0, 64) and M.combine(x, plan).shape == (0, 64)
    drows, dw = M.combine_grad(x, plan, torch.empty(0, 4, device=DEV), x)
    assert drows.shape == (0, 64) and dw.shape == (0, 4)


def _strided(rows, H, pad, dtype, seed, shift=0):
    """Rows of a wider tensor, `shift` elements into it."""
    g = torch.Generator().manual_seed(seed)
    store = torch.randn(rows, H + pad, generator=g).to(R.TYPES[dtype])
    return store[:, shift:shift + H], store.to(DEV)[:, shift:shift + H]


# (rows of 16, 8, 4 and 2 bytes' alignment; several to a block, one, several segments)
SHAPES = [(1, 4, 1, 64, 0, 0), (3, 8, 2, 1, 0, 0), (17, 9, 3, 130, 0, 0), (9, 5, 5, 1001, 0, 0),
          (6, 60, 4, 1024, 8, 0), (6, 60, 4, 1020, 4, 0), (5, 12, 8, 7168, 0, 0),
          (4, 40, 32, 257, 3, 1), (3, 6, 2, 20000, 0, 0)]


@pytest.mark.parametrize("T,E,K,H,pad,shift", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("empty", [0.0, 0.4])
def test_dispatch_combine_and_gradients(T, E, K, H, pad, shift, dtype, empty):
    dt = R.TYPES[dtype]
    ids = _ids(T, E, K, empty, H + T)
    if T > 2:
        ids[1] = -1 if empty else ids[1]  # a token without a route
    plan = M.sort_routes(ids.to(DEV), E)
    inv, n = plan.inv.cpu(), int(plan.n_rows)
    g = torch.Generator().manual_seed(H)
    w = torch.rand(T, K, generator=g)

    x, xc = _strided(T, H, pad, dtype, 1, shift)
    want = torch.full((T * K, H), 7.0, dtype=dt)
    for t in range(T):
        for k in range(K):
            if inv[t, k] >= 0:
                want[inv[t, k]] = x[t]
    rows_c = torch.full((T * K, H + pad), 7.0, dtype=dt, device=DEV)
    got = M.dispatch(xc, plan, rows=rows_c[:, shift:shift + H])
    assert torch.equal(got.cpu(), want)  # rows behind the last as they were
    rest = rows_c.clone()
    rest[:, shift:shift + H] = 7.0
    assert torch.all(rest == 7.0)  # and what lies between the rows

    rows, rc = _strided(T * K, H, pad, dtype, 2, shift)
    for weights in (w, None):
        out = M.combine(rc, plan, None if weights is None else weights.to(DEV)).cpu().double()
        want, mag = R.combine(rows, inv, weights)
        tol = R.half_step(dt) * want.abs() + 2 * K * 2.0 ** -24 * mag + R.tiny(dt)
        assert torch.all((out - want).abs() <= tol)

    dout, dc = _strided(T, H, pad, dtype, 3, shift)
    want, dw_want, mag = R.combine_grad(rows, inv, w, dout)
    drows, dw = M.combine_grad(rc, plan, w.to(DEV), dc,
                               drows=torch.full((T * K, H), 7.0, dtype=dt, device=DEV))
    err = (drows.cpu().double()[:n] - want[:n]).abs()
    assert torch.all(err <= (R.half_step(dt) + 2.0 ** -24) * want[:n].abs() + R.tiny(dt))
    assert torch.all(drows[n:] == 7.0)
    assert torch.all((dw.cpu().double() - dw_want).abs() <= (H / 32 + 64) * 2.0 ** -24 * mag)
    # over the rows themselves
    again, dw2 = M.combine_grad(rc, plan, w.to(DEV), dc, drows=rc)
    assert again is rc and torch.equal(again[:n], drows[:n]) and torch.equal(dw2, dw)


def test_gradients_against_differences():
    """<dout, combine(rows, w)> is linear in each weight and each row."""
    T, E, K, H = 6, 8, 3, 40
    ids = _ids(T, E, K, 0.2, 5)
    plan = M.sort_routes(ids.to(DEV), E)
    g = torch.Generator().manual_seed(6)
    rows = torch.randn(T * K, H, generator=g).to(DEV)
    w, dout = torch.rand(T, K, generator=g).to(DEV), torch.randn(T, H, generator=g).to(DEV)
    drows, dw = M.combine_grad(rows, plan, w, dout)

    def value(rows, w):
        return float((M.combine(rows, plan, w).double() * dout.double()).sum())

    for t in range(T):
        for k in range(K):
            step = torch.zeros_like(w)
            step[t, k] = 0.5
            diff = value(rows, w + step) - value(rows, w - step)
            assert abs(diff - float(dw[t, k])) <= 1e-4
            r = int(plan.inv[t, k])
            if r >= 0:
                step = torch.zeros_like(rows)
                step[r, 7] = 0.5
                diff = value(rows + step, w) - value(rows - step, w)
                assert abs(diff - float(drows[r, 7])) <= 1e-4


def test_special_values_stay_in_their_token():
    T, E, K, H = 4, 6, 2, 96
    ids = torch.tensor([[0, 1], [2, 3], [-1, 4], [5, -1]], dtype=torch.int32)
    plan = M.sort_routes(ids.to(DEV), E)
    rows = torch.ones(T * K, H, device=DEV)
    rows[int(plan.inv[0, 0]), 5] = float("nan")
    rows[int(plan.inv[1, 1]), 6] = float("inf")
    n = int(plan.n_rows)
    rows[n:] = float("nan")  # unused rows are not read
    w = torch.full((T, K), 0.5, device=DEV)
    w[2, 0] = float("nan")   # nor the weights of empty slots
    out = M.combine(rows, plan, w)
    assert torch.isnan(out[0, 5]) and torch.isinf(out[1, 6])
    assert int(torch.isfinite(out).logical_not().sum()) == 2
    drows, dw = M.combine_grad(rows, plan, w, torch.ones(T, H, device=DEV))
    assert torch.all(torch.isfinite(drows[:n])) and dw[2, 0] == 0 and dw[3, 1] == 0
    assert torch.isnan(dw[0, 0]) and torch.isinf(dw[1, 1]) and dw[0, 1] == H


def test_a_plan_that_is_none():
    """Row numbers outside [0, T*K) are empty slots, whoever made them."""
    T, K, H = 3, 2, 33
    inv = torch.tensor([[0, 6], [-5, 1 << 30], [5, 2]], dtype=torch.int32, device=DEV)
    plan = M.RoutePlan(torch.zeros(2, dtype=torch.int32, device=DEV),
                       torch.zeros(6, dtype=torch.int32, device=DEV), inv)
    x = torch.arange(T * H, dtype=torch.float32, device=DEV).reshape(T, H)
    rows = M.dispatch(x, plan, rows=torch.zeros(6, H, device=DEV))
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[5], x[2])
    assert torch.equal(M.combine(rows, plan)[1], torch.zeros(H, device=DEV))
    _, dw = M.combine_grad(rows, plan, torch.ones(T, K, device=DEV), x)
    assert dw[1].tolist() == [0.0, 0.0] and dw[0, 1] == 0


def test_rows_more_than_32_bits_apart():
    """Rows whose last elements lie past 2^31 elements (and 2^32 bytes)."""
    T, E, K, ld = 90, 16, 4, 8_000_000
    for H in (64, 33):  # by 16 bytes, by the element
        plan = M.sort_routes(_ids(T, E, K, 0.1, 3).to(DEV), E)
        n = int(plan.n_rows)
        x = torch.randn(T, H, device=DEV).bfloat16()
        w = torch.rand(T, K, device=DEV)
        store = torch.empty(T * K * ld, dtype=torch.bfloat16, device=DEV)
        far = torch.as_strided(store, (T * K, H), (ld, 1))
        rows = M.dispatch(x, plan)
        assert torch.equal(M.dispatch(x, plan, rows=far)[:n], rows[:n])
        assert torch.equal(M.combine(far, plan, w), M.combine(rows, plan, w))
        drows, dw = M.combine_grad(rows, plan, w, x)
        got, dw2 = M.combine_grad(far, plan, w, x, drows=far)
        assert torch.equal(got[:n], drows[:n]) and torch.equal(dw2, dw)


def test_graph_stream_and_repeat():
    T, E, K, H = 700, 64, 8, 512
    ids = _ids(T, E, K, 0.1, 8).to(DEV)
    x = torch.randn(T, H, device=DEV).bfloat16()
    w = torch.rand(T, K, device=DEV)

    def run():
        plan = M.sort_routes(ids, E)
        rows = M.dispatch(x, plan, rows=torch.zeros(T * K, H, dtype=x.dtype, device=DEV))
        out = M.combine(rows, plan, w)
        drows, dw = M.combine_grad(rows, plan, w, out,
                                   drows=torch.zeros_like(rows))
        return [plan.offsets, plan.perm, plan.inv, rows, out, drows, dw]

    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = run()
    ids.copy_(torch.flip(ids, [0]))
    graph.replay()
    fresh = run()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    for a, b in zip(third, fresh):
        assert torch.equal(a, b)


def test_refusals():
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    plan = M.sort_routes(ids, 3)
    x = torch.zeros(4, 8, device=DEV)
    for bad in (lambda: M.sort_routes(ids.cpu(), 3), lambda: M.sort_routes(ids[0], 3),
                lambda: M.sort_routes(ids.float(), 3), lambda: M.dispatch(x[:3], plan),
                lambda: M.dispatch(x.t(), plan), lambda: M.dispatch(x.double(), plan),
                lambda: M.dispatch(x.cpu(), plan),
                lambda: M.dispatch(x, plan, rows=torch.zeros(8, 8, device=DEV).half()),
                lambda: M.dispatch(x, plan, rows=torch.zeros(7, 8, device=DEV)),
                lambda: M.combine(torch.zeros(8, 8, device=DEV), plan, torch.ones(4, 3, device=DEV)),
                lambda: M.combine_grad(torch.zeros(8, 8, device=DEV), plan, None, x[:, :4]),
                lambda: M.dispatch(x, M.RoutePlan(plan.offsets, plan.perm, plan.inv.long()))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(M.MoeError):
        M.combine(x, plan)  # 4 rows for 8 routes
    with pytest.raises(M.MoeError):
        M.sort_routes(ids, 1)  # K > E
    with pytest.raises(M.MoeError):
        M.sort_routes(ids, 3, ws=torch.empty(128, dtype=torch.uint8, device=DEV))
