"""Rows kept in 8 bits and the experts' activation with its gradient from them, against
plain definitions in 64 bits.

Bounds: what is kept is exact.  The activation's fp32 arithmetic is off by (8 + 1.2 |g|) 2^-23
of the result at most (fast exponential 2 + 1.17 |g| units, quotient 2, products), its
gradient by (12 + 4 |g|) 2^-23 of its terms' magnitudes (s is off by (5 + 1.2 |g|) 2^-23 of
itself, 1 - s by 3 2^-23, which g multiplies); then one rounding.
Below exp's range (g < -87) s is under 2^-126 and may be 0.
"""
import math

import pytest
import torch

import nvfp4_token_routed_gb300 as M
import expert_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _values(rows, cols, dtype, seed, pad=0, shift=0):
    """Rows over many magnitudes, some zeros, views of a wider tensor."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g)
    x *= torch.exp2(torch.randint(-6, 4, (rows, 1), generator=g).float())
    x[:, ::7] *= 20.0
    x[torch.rand(x.shape, generator=g) < 0.05] = 0.0
    x = x.to(R.TYPES[dtype])
    return x[:, shift:shift + cols], x.to(DEV)[:, shift:shift + cols]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (3, 31, 0, 0), (2, 32, 0, 0),
                                                 (5, 33, 1, 1), (7, 100, 4, 0), (4, 256, 8, 0),
                                                 (9, 1407, 0, 0), (3, 7168, 0, 0)])
def test_checkpoint_round_trip(rows, cols, pad, shift, dtype):
    x, xc = _values(rows, cols, dtype, rows + cols, pad, shift)
    kept = M.checkpoint(xc)
    want, byte = R.held8(x)
    assert torch.equal(kept.scales.cpu()[:, 0], byte)
    got = M.restore(kept, torch.float32)
    assert torch.equal(got.cpu().double(), want)
    assert torch.equal(M.restore(kept).cpu(), want.to(R.TYPES[dtype]))
    wide = torch.full((rows, cols + 3), 5.0, dtype=R.TYPES[dtype], device=DEV)
    M.restore(kept, out=wide[:, 1:1 + cols], dtype=R.TYPES[dtype])
    assert torch.equal(wide[:, 1:1 + cols].cpu(), want.to(R.TYPES[dtype]))
    assert torch.all(wide[:, 0] == 5.0) and torch.all(wide[:, 1 + cols:] == 5.0)
    # half a step of the element, or of the block's smallest
    unit = torch.exp2(byte.double() - 127).repeat_interleave(32, 1)[:, :cols]
    assert torch.all((want - x.double()).abs() <= torch.maximum(2.0 ** -4 * x.double().abs(),
                                                                unit * 2.0 ** -10))


def test_block_borders_and_special_values():
    x = torch.zeros(12, 32)
    top = [448.0, 449.0, 448.0 * 2 ** 60, 1.75, 1.7500001, 2.0 ** -126, 2.0 ** -149, 3.3e38, 0.0,
           math.inf, math.nan, -448.0]
    for i, v in enumerate(top):
        x[i, 0] = v
        x[i, 1] = v / 3 if math.isfinite(v) else 1.0
    kept = M.checkpoint(x.to(DEV))
    want, byte = R.held8(x)
    assert torch.equal(kept.scales.cpu()[:, 0], byte)
    got = M.restore(kept).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(want).sum() == 64
    same = torch.equal(got.nan_to_num().double(), want.nan_to_num())
    assert same
    assert float(got[0, 0]) == 448.0 and float(got[11, 0]) == -448.0 and float(got[7, 0]) == 240.0 * 2.0 ** 120


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_the_types_largest_values_stay_finite(dtype):
    info = torch.finfo(R.TYPES[dtype])
    x = torch.tensor([info.max, info.min, 0.98 * info.max, 0.9 * info.max, -1.0, 0.5 * info.max])
    x = x.to(R.TYPES[dtype]).repeat(2, 12)  # blocks of 32 and a part
    want, byte = R.held8(x)
    kept = M.checkpoint(x.to(DEV))
    got = M.restore(kept).cpu()
    assert torch.all(torch.isfinite(got)) and torch.equal(got.double(), want)
    assert torch.all((got.double() - x.double()).abs() <= x.double().abs() / 16 + 2.0 ** -10 *
                     torch.exp2(byte.double().max() - 127))
    h = torch.cat([x, torch.ones_like(x)], 1).to(DEV)  # the lowest gate gives 0, and no gradient
    y, kept = M.expert_act(h, "swiglu", checkpoint=True)
    dh = M.expert_act_grad(kept, torch.ones_like(y))
    assert torch.all(y[:, 1::6] == 0) and torch.all(dh[:, 1:72:6] == 0)
    assert torch.all(torch.isfinite(dh))


def test_outputs_of_another_type():
    x = torch.randn(3, 40, device=DEV).bfloat16()
    out = torch.empty(3, 40, device=DEV)
    assert M.restore(M.checkpoint(x), out=out) is out
    assert torch.equal(out.bfloat16(), M.restore(M.checkpoint(x)))
    assert M.mx_restore(M.mx_quantize(x), out=out) is out
    assert torch.equal(out.bfloat16(), M.mx_restore(M.mx_quantize(x)))


ACTS = [("swiglu", 0.0), ("swiglu", 1.5), ("relu2", 0.0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act,limit", ACTS)
@pytest.mark.parametrize("rows,I,pad,shift", [(1, 1, 0, 0), (2, 33, 0, 0), (5, 64, 2, 0),
                                              (3, 100, 4, 0), (4, 1024, 0, 0), (6, 703, 1, 1)])
def test_activation_and_gradient(rows, I, pad, shift, act, limit, dtype):
    dt = R.TYPES[dtype]
    halves = 2 if act == "swiglu" else 1
    h, hc = _values(rows, halves * I, dtype, I, pad, shift)
    y, kept = M.expert_act(hc, act, limit, checkpoint=True)
    assert torch.equal(M.expert_act(hc, act, limit), y)
    want = R.act(h, act, limit)
    g = h[:, :I].double().abs()
    tol = (R.half_step(dt) + (8 + 1.2 * g) * 2.0 ** -23) * want.abs() + R.tiny(dt)
    if act == "swiglu":
        tol = tol + 2.0 ** -125 * (g * h[:, I:].double()).abs()
    big = want.abs() > torch.finfo(dt).max  # fp16 squares
    assert torch.all(((y.cpu().double() - want).abs() <= tol) | big)

    dy, dc = _values(rows, I, dtype, I + 1, pad, shift)
    wide = torch.full((rows, halves * I + pad), 7.0, dtype=dt, device=DEV)
    dh = M.expert_act_grad(kept, dc, dh=wide[:, shift:shift + halves * I])
    rest = wide.clone()
    rest[:, shift:shift + halves * I] = 7.0
    assert torch.all(rest == 7.0)
    want, weight = R.act_grad(R.kept(h, act), act, limit, dy)
    tol = R.half_step(dt) * want.abs() + 2.0 ** -23 * weight + R.tiny(dt)
    big = want.abs() > torch.finfo(dt).max
    assert torch.all(((dh.cpu().double() - want).abs() <= tol) | big)
    assert torch.equal(M.expert_act_grad(kept, dc).cpu(), dh.cpu())


@pytest.mark.parametrize("act,limit", ACTS)
def test_gradient_against_differences(act, limit):
    """Where h is held exactly, the gradient is the activation's slope."""
    I, halves = 64, 2 if act == "swiglu" else 1
    g = torch.Generator().manual_seed(3)
    h = torch.randint(-14, 15, (4, halves * I), generator=g).float() / 4 + 0.125
    h = R.kept(h, act).float()
    assert torch.equal(R.kept(h, act).float(), h)
    dy = torch.randn(4, I, generator=g)
    _, kept = M.expert_act(h.to(DEV), act, limit, checkpoint=True)
    dh = M.expert_act_grad(kept, dy.to(DEV)).cpu().double()
    step = 1e-5
    for j in range(0, halves * I, 5):
        d = torch.zeros(h.shape, dtype=torch.float64)
        d[:, j] = step
        diff = (R.act(h.double() + d, act, limit) - R.act(h.double() - d, act, limit)) / (2 * step)
        want = (diff * dy.double()).sum(1)
        # limits of 1.5 are met exactly by some values: one-sided there
        free = ((h[:, j].double().abs() - limit).abs() > 1e-3) if limit else torch.ones(4).bool()
        assert torch.all(((dh[:, j] - want).abs() <= 1e-4 + 1e-4 * want.abs())[free])


def test_limit_itself_passes():
    h = torch.tensor([[1.5, 2.0, 1.5, 1.5], [1.0, 1.5, -1.5, -2.0]]).reshape(1, 8).to(DEV)
    _, kept = M.expert_act(h, "swiglu", 1.5, checkpoint=True)
    dh = M.expert_act_grad(kept, torch.ones(1, 4, device=DEV))[0]
    assert (dh != 0).tolist() == [True, False, True, True, True, True, True, False]


def test_special_values_stay_in_their_block():
    h = torch.ones(2, 128, device=DEV)
    h[0, 3], h[1, 70] = float("nan"), float("inf")
    y, kept = M.expert_act(h, "swiglu", checkpoint=True)
    assert torch.isnan(y[0, 3]) and torch.isinf(y[1, 6])
    assert int(torch.isfinite(y).logical_not().sum()) == 2
    dh = M.expert_act_grad(kept, torch.ones(2, 64, device=DEV))
    bad = torch.isfinite(dh).logical_not()
    assert torch.all(bad[0, :32]) and torch.all(bad[0, 64:96]) and not bad[0, 32:64].any()
    assert torch.all(bad[1, :32]) and not bad[1, 32:64].any() and not bad[1, 96:].any()
    low = torch.full((1, 64), torch.finfo(torch.float32).min, device=DEV)
    assert torch.all(torch.isfinite(M.expert_act(low, "swiglu")).logical_not() |
                     (M.expert_act(low, "swiglu").abs() <= 0))
    assert torch.equal(M.expert_act(low, "relu2"), torch.zeros(1, 64, device=DEV))


def test_rows_more_than_32_bits_apart():
    R_, ld = 300, 8_000_000
    store = torch.empty(R_ * ld, dtype=torch.bfloat16, device=DEV)
    for W in (128, 66):
        _, x = _values(R_, W, "bf16", W)
        far = torch.as_strided(store, (R_, W), (ld, 1))
        far.copy_(x)
        kept, want = M.checkpoint(far), M.checkpoint(x)
        assert torch.equal(kept.codes, want.codes) and torch.equal(kept.scales, want.scales)
        assert torch.equal(M.restore(kept, out=far), M.restore(want))
        far.copy_(x)
        y, k1 = M.expert_act(far, "swiglu", checkpoint=True)
        y2, k2 = M.expert_act(x, "swiglu", checkpoint=True)
        assert torch.equal(y, y2) and torch.equal(k1.codes, k2.codes)
        assert torch.equal(M.expert_act_grad(k1, y, dh=far), M.expert_act_grad(k2, y2))


def test_many_short_and_long_rows():
    """Spans several to a warp and one, many rows to a block and many blocks to a row."""
    for R_, W in ((5000, 40), (3000, 1031), (40, 20000), (1, 300000)):
        _, x = _values(R_, 2 * W, "bf16", W)
        y, kept = M.expert_act(x, "swiglu", checkpoint=True)
        gate, up = x[:, :W].float(), x[:, W:].float()
        want = (gate.double() * torch.sigmoid(gate.double()) * up.double())
        g = gate.abs().double()
        tol = (R.half_step(torch.bfloat16) + (8 + 1.2 * g) * 2.0 ** -23) * want.abs() + 2.0 ** -125 * g * up.abs()
        assert torch.all((y.double() - want).abs() <= tol + R.tiny(torch.bfloat16))
        halves = torch.cat([M.restore(M.checkpoint(h.contiguous()), torch.float32)
                            for h in (x[:, :W], x[:, W:])], 1).double()
        dh = M.expert_act_grad(kept, y).double()
        want, weight = R.act_grad(halves, "swiglu", 0.0, y)
        tol = R.half_step(torch.bfloat16) * want.abs() + 2.0 ** -23 * weight
        assert torch.all((dh - want).abs() <= tol + R.tiny(torch.bfloat16))


@pytest.mark.parametrize("n", [0, 1, 5, 9, 50])
def test_rows_behind_the_last(n):
    """n_rows on the device: rows from there on are neither read nor written."""
    x = torch.randn(9, 96, device=DEV)
    count = torch.tensor([n], dtype=torch.int32, device=DEV)
    kept = M.Checkpoint(*[torch.full(s, 9, dtype=torch.uint8, device=DEV)
                          for s in ((9, 1, 96), (9, 1, 3))], 96, x.dtype, None, 0.0)
    M.checkpoint(x, kept=kept, n_rows=count)
    n = min(n, 9)
    assert torch.all(kept.codes[n:] == 9) and torch.all(kept.scales[n:] == 9)
    assert torch.equal(kept.codes[:n], M.checkpoint(x).codes[:n])
    out = M.restore(kept, out=torch.full((9, 96), 7.0, device=DEV), n_rows=count)
    assert torch.all(out[n:] == 7.0)
    y = torch.full((9, 48), 7.0, device=DEV)
    _, k2 = M.expert_act(x, "swiglu", checkpoint=True, y=y, n_rows=count)
    assert torch.all(y[n:] == 7.0) and torch.equal(y[:n], M.expert_act(x, "swiglu")[:n])
    dh = M.expert_act_grad(k2, y, dh=torch.full((9, 96), 7.0, device=DEV), n_rows=count)
    assert torch.all(dh[n:] == 7.0)


def test_no_rows_and_refusals():
    x = torch.empty(0, 64, device=DEV)
    assert M.restore(M.checkpoint(x)).shape == (0, 64)
    y, kept = M.expert_act(x, "swiglu", checkpoint=True)
    assert y.shape == (0, 32) and M.expert_act_grad(kept, y).shape == (0, 64)
    h = torch.zeros(4, 64, device=DEV)
    _, kept = M.expert_act(h, "swiglu", checkpoint=True)
    for bad in (lambda: M.checkpoint(h.cpu()), lambda: M.checkpoint(h.t()),
                lambda: M.checkpoint(h.double()), lambda: M.restore(kept),
                lambda: M.expert_act_grad(M.checkpoint(h), h),
                lambda: M.expert_act_grad(kept, h), lambda: M.expert_act_grad(kept, h[:3, :32]),
                lambda: M.expert_act(h, "swiglu", kept=M.checkpoint(h)),
                lambda: M.expert_act(h, "relu2", kept=kept), lambda: M.expert_act(h, "gelu"),
                lambda: M.expert_act(h, "swiglu", n_rows=torch.zeros(1, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: M.expert_act(h, "relu2", 1.0), lambda: M.expert_act(h, "swiglu", -1.0),
                lambda: M.expert_act(h, "swiglu", float("nan")),
                lambda: M.expert_act(h[:, :63], "swiglu", y=torch.zeros(4, 31, device=DEV))):
        with pytest.raises(M.MoeError):
            bad()
