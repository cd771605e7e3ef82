"""Microscaled FP4: quantisation (exact) and products, against plain definitions in 64 bits.

Bound of a product: both operands' values are exact in the product's definition; the fp32
accumulator takes D / 64 instructions, each off by at most 2^-22 of what it holds, which is
at most the sum of the terms' magnitudes; then one rounding.
"""
import math

import pytest
import torch

import nvfp4_token_routed_gb300 as M
import expert_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _values(rows, cols, dtype, seed, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g)
    x *= torch.exp2(torch.randint(-4, 5, (rows, 1), generator=g).float())
    x[torch.rand(x.shape, generator=g) < 0.05] = 0.0
    x = x.to(R.TYPES[dtype])
    return x[:, shift:shift + cols], x.to(DEV)[:, shift:shift + cols]


def _scales(q, rows, cols):
    """Scale bytes [rows, blocks] from the panels."""
    return q.scales.cpu().permute(1, 0, 2).reshape(q.scales.shape[1], -1)[:rows,
                                                                         :(cols + 31) // 32]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (2, 32, 0, 0), (3, 100, 4, 0),
                                                 (5, 257, 1, 1), (4, 512, 8, 0), (7, 801, 0, 0),
                                                 (2, 2048, 0, 0)])
def test_quantize(rows, cols, pad, shift, dtype):
    x, xc = _values(rows, cols, dtype, rows + cols, pad, shift)
    q = M.mx_quantize(xc)
    want, byte = R.held4(x)
    assert torch.equal(_scales(q, rows, cols), byte)
    assert torch.equal(M.mx_restore(q, torch.float32).cpu().double(), want)
    assert torch.equal(M.mx_restore(q, x.dtype).cpu(), want.to(x.dtype))
    codes = q.codes.cpu()
    nibbles = torch.stack([codes & 15, codes >> 4], 2).reshape(rows, -1)
    value = R.E2M1[(nibbles & 7).long()] * torch.where(nibbles >= 8, -1.0, 1.0)
    unit = torch.exp2(byte.double() - 127).repeat_interleave(32, 1)[:, :cols]
    assert torch.equal(value[:, :cols] * unit, want) and not nibbles[:, cols:].any()
    # half a step of the element, or of the block's smallest
    assert torch.all((want - x.double()).abs() <=
                     torch.maximum(x.double().abs() / 4, unit / 4))


def test_quantize_borders_and_special_values():
    x = torch.zeros(12, 32)
    top = [6.0, 6.0000005, 5.0, 2.5, 3.5, 1.5, 2.0 ** -130, 3.3e38, 0.0, math.inf, math.nan, -6.0]
    for i, v in enumerate(top):
        x[i, 0] = v
        x[i, 1:8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * (v / 6 if
                                                                            math.isfinite(v) else 1)
    q = M.mx_quantize(x.to(DEV))
    want, byte = R.held4(x)
    assert torch.equal(_scales(q, 12, 32), byte)
    got = M.mx_restore(q, torch.float32).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and int(torch.isnan(got).sum()) == 64
    # the value next to the type's largest rounds to 2^128, which fp32 writes as infinity
    same = torch.equal(got.nan_to_num(), want.float().nan_to_num())
    assert same


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,D,C", [(1, 1, 1), (3, 33, 40), (2, 300, 65), (5, 512, 32)])
def test_quantize_transposed(E, D, C, dtype):
    g = torch.Generator().manual_seed(D)
    x = torch.randn(E, D, C, generator=g).to(R.TYPES[dtype]).to(DEV)
    q, want = M.mx_quantize_transposed(x), M.mx_quantize(x.transpose(1, 2).contiguous())
    assert q.shape == want.shape == (E, C, D) and torch.equal(q.codes, want.codes)
    assert torch.equal(q.scales[:, :E * C], want.scales[:, :E * C])
    one = M.mx_quantize_transposed(x[0])
    assert one.shape == (C, D) and torch.equal(one.codes, q.codes[:C])


def _product(x, w, offsets, dtype, out=None):
    """x [R, D], w [E, N, D] on the CPU: checks the library's product of their MX forms."""
    E, N, D = w.shape
    q, qw = M.mx_quantize(x.to(DEV)), M.mx_quantize(w.to(DEV))
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    got = M.mx_product(q, qw, off, dtype, out=out)
    xv, wv = M.mx_restore(q, torch.float32).double(), M.mx_restore(qw, torch.float32).double()
    cuts = [0, x.shape[0]] if offsets is None else offsets
    for e in range(E):
        a, b = cuts[e], cuts[e + 1]
        if a == b:
            continue
        want = xv[a:b] @ wv[e].t()
        mag = xv[a:b].abs() @ wv[e].abs().t()
        tol = R.half_step(dtype) * want.abs() + (D / 64 + 4) * 2.0 ** -22 * mag + R.tiny(dtype)
        bad = (got[a:b].double() - want).abs() > tol
        assert not bad.any(), (e, bad.nonzero()[:4].tolist(), int(bad.sum()))
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R_,N,D", [(1, 1, 1), (1, 128, 256), (16, 256, 512), (17, 130, 300),
                                    (128, 384, 256), (129, 127, 1000), (192, 512, 256),
                                    (193, 64, 2048), (400, 1003, 801), (1000, 2048, 64)])
def test_product_of_one_matrix(R_, N, D, dtype):
    x, _ = _values(R_, D, "bf16", R_ + D)
    w = torch.randn(1, N, D, generator=torch.Generator().manual_seed(N)) * D ** -0.5
    _product(x, w, None, R.TYPES[dtype])


GROUPS = [[0, 3, 3, 4, 20], [0, 0, 0, 0, 1], [0, 64, 128, 193, 194], [0, 193, 386, 386, 1100],
          [0, 16, 33, 47, 400]]


@pytest.mark.parametrize("offsets", GROUPS)
@pytest.mark.parametrize("N,D", [(128, 256), (257, 700), (96, 2304)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product_of_groups(offsets, N, D, dtype):
    E, rows = len(offsets) - 1, offsets[-1]
    x, _ = _values(rows, D, "f32", rows)
    w = torch.randn(E, N, D, generator=torch.Generator().manual_seed(N)) * D ** -0.5
    _product(x, w, offsets, R.TYPES[dtype])


def test_many_experts_and_items():
    g = torch.Generator().manual_seed(9)
    load = torch.randint(0, 9, (1024,), generator=g)
    load[torch.rand(1024, generator=g) < 0.5] = 0
    offsets = [0] + load.cumsum(0).tolist()
    x, _ = _values(offsets[-1], 256, "bf16", 3)
    _product(x, torch.randn(1024, 129, 256, generator=g) / 16, offsets, torch.bfloat16)


def test_rows_outside_the_groups_and_between_rows():
    """Groups that leave rows out, an output of strided rows, and offsets past the last row."""
    x, _ = _values(50, 256, "bf16", 5)
    w = torch.randn(3, 40, 256) / 16
    for pad in (0, 1, 6):
        store = torch.full((50, 40 + pad), 7.0, dtype=torch.bfloat16, device=DEV)
        got = _product(x, w, [5, 9, 9, 41], torch.bfloat16, out=store[:, pad:])
        assert torch.all(got[:5] == 7.0) and torch.all(got[41:] == 7.0)
        assert torch.all(store[:, :pad] == 7.0)
    q, qw = M.mx_quantize(x.to(DEV)), M.mx_quantize(w.to(DEV))
    bad = torch.tensor([-7, 9, 9, 1000], dtype=torch.int32, device=DEV)
    good = torch.tensor([0, 9, 9, 50], dtype=torch.int32, device=DEV)
    assert torch.equal(M.mx_product(q, qw, bad), M.mx_product(q, qw, good))


@pytest.mark.parametrize("rows,N,D,offsets", [(50, 40, 256, [3, 20, 5, 33]),
                                              (2048, 1300, 2048, [100, 1500, 200, 2000])])
def test_offsets_that_do_not_ascend(rows, N, D, offsets):
    """Rows of one group alone are its product, and no row is written outside the groups."""
    x, _ = _values(rows, D, "bf16", N)
    w = torch.randn(3, N, D, generator=torch.Generator().manual_seed(D)) / D ** 0.5
    q, qw = M.mx_quantize(x.to(DEV)), M.mx_quantize(w.to(DEV))
    out = torch.full((rows + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    M.mx_product(q, qw, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=out[1:-1])
    a, b, c, d = offsets
    first, last = (M.mx_product(q, qw, torch.tensor(o, dtype=torch.int32, device=DEV))
                   for o in ([a, b, b, b], [c, c, c, d]))
    got = out[1:-1]
    assert torch.equal(got[a:c], first[a:c]) and torch.equal(got[b:d], last[b:d])
    assert torch.all(out[:a + 1] == 7.0) and torch.all(out[d + 1:] == 7.0)


def test_a_row_does_not_depend_on_its_batch():
    x, _ = _values(300, 1024, "bf16", 6)
    w = torch.randn(2, 200, 1024) / 32
    qw = M.mx_quantize(w.to(DEV))
    off = torch.tensor([0, 190, 300], dtype=torch.int32, device=DEV)
    whole = M.mx_product(M.mx_quantize(x.to(DEV)), qw, off)
    for a, b in ((0, 1), (7, 40), (189, 192), (250, 300)):
        part = M.mx_quantize(x[a:b].contiguous().to(DEV))
        o = torch.tensor([0, max(0, min(b, 190) - a), b - a], dtype=torch.int32, device=DEV)
        assert torch.equal(M.mx_product(part, qw, o), whole[a:b])


def test_non_finite_blocks_stay_in_their_row():
    x, _ = _values(20, 256, "f32", 7)
    x = x.clone()
    x[3, 40], x[11, 5] = math.nan, math.inf
    w = torch.randn(70, 256) / 16
    w[9, 200] = math.inf
    y = M.mx_product(M.mx_quantize(x.to(DEV)), M.mx_quantize(w.to(DEV)), dtype=torch.float32)
    bad = torch.isnan(y)
    want = torch.zeros(20, 70, dtype=torch.bool, device=DEV)
    want[3], want[11], want[:, 9] = True, True, True
    assert torch.equal(bad, want)


def test_dispatch_of_quantised_rows():
    for T, E, K, D in ((1, 4, 1, 40), (9, 8, 3, 300), (40, 12, 5, 512)):
        ids = torch.rand(T, E).argsort(1)[:, :K].int()
        ids[torch.rand(T, K) < 0.2] = -1
        plan = M.sort_routes(ids.to(DEV), E)
        _, xc = _values(T, D, "bf16", T)
        got = M.dispatch(M.mx_quantize(xc), plan)
        want = M.mx_quantize(M.dispatch(xc, plan))
        n = int(plan.n_rows)
        assert got.shape == (T * K, D) and torch.equal(got.codes[:n], want.codes[:n])
        assert torch.equal(got.scales[:, :n], want.scales[:, :n])


@pytest.mark.parametrize("n", [0, 3, 8, 30])
def test_rows_behind_the_last(n):
    x = torch.randn(8, 300, device=DEV)
    count = torch.tensor([n], dtype=torch.int32, device=DEV)
    q = M.MxTensor.empty((8, 300), x)
    q.codes.fill_(9), q.scales.fill_(9)
    M.mx_quantize(x, out=q, n_rows=count)
    n = min(n, 8)
    full = M.mx_quantize(x)
    assert torch.equal(q.codes[:n], full.codes[:n]) and torch.all(q.codes[n:] == 9)
    assert torch.equal(q.scales[:, :n], full.scales[:, :n]) and torch.all(q.scales[:, n:] == 9)
    out = M.mx_restore(full, torch.float32, out=torch.full((8, 300), 7.0, device=DEV), n_rows=count)
    assert torch.all(out[n:] == 7.0)


def test_graphs_and_streams_need_no_workspace():
    """Two captured products replayed on two streams at once."""
    x, xc = _values(333, 512, "bf16", 8)
    w = M.mx_quantize(torch.randn(4, 256, 512, device=DEV) / 22)
    off = torch.tensor([0, 100, 101, 300, 333], dtype=torch.int32, device=DEV)
    want = M.mx_product(M.mx_quantize(xc), w, off)
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(M.mx_product(M.mx_quantize(xc), w, off))
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_no_rows_and_refusals():
    x = torch.randn(4, 64, device=DEV)
    q, w = M.mx_quantize(x), M.mx_quantize(torch.randn(2, 8, 64, device=DEV))
    empty = M.mx_quantize(torch.empty(0, 64, device=DEV))
    assert M.mx_product(empty, w, torch.zeros(3, dtype=torch.int32, device=DEV)).shape == (0, 8)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    for bad in (lambda: M.mx_quantize(x.cpu()), lambda: M.mx_quantize(x.t()),
                lambda: M.mx_quantize(x.double()), lambda: M.mx_quantize(x[0]),
                lambda: M.mx_product(q, w), lambda: M.mx_product(q, w, off[:2]),
                lambda: M.mx_product(q, w, off.long()), lambda: M.mx_product(w, w, off),
                lambda: M.mx_product(q, w, off, out=torch.zeros(4, 9, device=DEV)),
                lambda: M.mx_product(q, w, off, dtype=torch.float64),
                lambda: M.mx_quantize(x, out=w),
                lambda: M.mx_product(M.MxTensor(q.codes[:, :64], q.scales, (4, 64)), w, off),
                lambda: M.mx_quantize_transposed(x.t())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(M.MoeError):
        M.mx_product(M.mx_quantize(torch.randn(4, 65, device=DEV)), w, off)


def test_long_rows():
    """The longest reduction (256 stages) and rows of the most outputs."""
    x, _ = _values(3, 65536, "bf16", 11)
    w = torch.randn(1, 130, 65536, generator=torch.Generator().manual_seed(1)) / 256
    _product(x, w, None, torch.bfloat16)
    x, _ = _values(5, 40, "bf16", 12)
    _product(x, torch.randn(1, 65536, 40, generator=torch.Generator().manual_seed(2)) / 6, None,
             torch.float16)


def test_outputs_more_than_32_bits_apart():
    """Rows of an output whose last elements lie past 2^31 elements (and 2^32 bytes)."""
    R_, N, ld = 300, 260, 8_000_000
    x, xc = _values(R_, 256, "bf16", 13)
    w = M.mx_quantize(torch.randn(N, 256, device=DEV) / 16)
    q = M.mx_quantize(xc)
    want = M.mx_product(q, w)
    store = torch.empty(R_ * ld, dtype=torch.bfloat16, device=DEV)
    for shift in (0, 1):  # stores of 8 bytes, and by the element
        out = torch.as_strided(store, (R_, N), (ld, 1), shift)
        assert torch.equal(M.mx_product(q, w, out=out), want)
    few = M.mx_product(M.mx_quantize(xc[:40].contiguous()), w,
                       out=torch.as_strided(store, (40, N), (50_000_000, 1)))
    assert torch.equal(few, want[:40])
    far = torch.as_strided(store, (R_, 256), (ld, 1))
    far.copy_(xc)
    again = M.mx_quantize(far)
    assert torch.equal(again.codes, q.codes) and torch.equal(again.scales, q.scales)
    assert torch.equal(M.mx_restore(q, out=far), M.mx_restore(q))


# rows an expert, experts, outputs, length: pairs of blocks take these (stages from 8 on, 38
# items or more of 256 rows and outputs); row tiles of 32 to 256 rows, one and two accumulators
@pytest.mark.parametrize("rows,E,N,D", [(229, 5, 2436, 2048), (256, 4, 2560, 2100),
                                        (257, 4, 2561, 2048), (288, 4, 2499, 1999),
                                        (500, 2, 3301, 2305), (1023, 1, 2818, 4001),
                                        (160, 9, 2305, 1900)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_product_by_pairs_of_blocks(rows, E, N, D, dtype):
    offsets = [0] + [3 + rows * (i + 1) for i in range(E)]
    offsets[-1] += 224 * E - min(224 * E, offsets[-1])
    x, _ = _values(offsets[-1], D, "bf16", rows)
    w = torch.randn(E, N, D, generator=torch.Generator().manual_seed(N)) * D ** -0.5
    _product(x, w, offsets, R.TYPES[dtype])


def test_ragged_groups_by_pairs_of_blocks():
    offsets = [0, 1, 1, 700, 731, 1060, 1500, 1500, 2001]
    x, _ = _values(2001, 2048, "bf16", 4)
    w = torch.randn(8, 1400, 2048, generator=torch.Generator().manual_seed(4)) / 45
    store = torch.full((2001, 1401), 7.0, dtype=torch.bfloat16, device=DEV)
    for out in (None, store[:, 1:], torch.as_strided(store, (2001, 1400), (1401, 1))):
        _product(x, w, offsets, torch.bfloat16, out=out)


def test_a_row_has_the_same_bits_in_pairs():
    x, _ = _values(2000, 2048, "bf16", 15)
    w = M.mx_quantize(torch.randn(1, 1300, 2048, device=DEV) / 45)
    whole = M.mx_product(M.mx_quantize(x.to(DEV)), w)
    for a, b in ((0, 1), (777, 900), (1990, 2000)):
        part = M.mx_product(M.mx_quantize(x[a:b].contiguous().to(DEV)), w)
        assert torch.equal(part, whole[a:b])


def test_expired_waits_give_nan_in_pairs():
    x, xc = _values(1000, 2048, "bf16", 14)
    w = M.mx_quantize(torch.randn(2, 3328, 2048, device=DEV) / 45)
    off = torch.tensor([0, 501, 1000], dtype=torch.int32, device=DEV)
    q = M.mx_quantize(xc)
    want = M.mx_product(q, w, off)
    # expert 1 has items 26 .. 51: its second row tile of outputs 256 .. 511
    got = M.moe_nvfp4_selftest_product_timeout(q, w, off, 29)
    lost = torch.isnan(got)
    assert torch.all(lost[757:, 256:512]) and int(lost.sum()) == 243 * 256
    assert torch.equal(got[~lost], want[~lost])
    assert torch.equal(M.mx_product(q, w, off), want)


def test_expired_waits_give_nan():
    """Row loads that leave before an item: its block's items from there on get NaN, the
    rest their results, and the context stays usable."""
    x, xc = _values(40, 512, "bf16", 10)
    w = M.mx_quantize(torch.randn(2, 384, 512, device=DEV) / 22)
    off = torch.tensor([0, 17, 40], dtype=torch.int32, device=DEV)
    q = M.mx_quantize(xc)
    want = M.mx_product(q, w, off)
    got = M.moe_nvfp4_selftest_product_timeout(q, w, off, 4)  # expert 1, its second weight tile
    lost = torch.isnan(got)
    assert torch.all(lost[17:, 128:256]) and int(lost.sum()) == 23 * 128
    assert torch.equal(got[~lost], want[~lost])
    assert torch.equal(M.mx_product(q, w, off), want)
