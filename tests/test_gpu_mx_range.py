"""Microscaled FP4 at the end of the types' ranges: a value rounds to the nearest code also
where that passes its type's largest, products take it as what it stands for, and only
restoring to a type that ends before gives an infinity."""
import math

import pytest
import torch

import nvfp4_token_routed_gb300 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _nearest(v):
    """The E2M1 value times a power of two that v > 0, alone in its block, is held as."""
    e = math.frexp(v / 6.0)[1] - 1  # smallest e with v <= 6 * 2^e
    e = e + 1 if v > 6.0 * 2.0 ** e else e
    # 3 to 6 units: steps of 1 below 4, of 2 from there on; ties to the even code
    u = v / 2.0 ** e
    near = {3: 3.0, 4: 4.0, 5: 4.0, 6: 6.0}
    return near[round(u)] * 2.0 ** e if u < 4.0 else (4.0 if u <= 5.0 else 6.0) * 2.0 ** e


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_values_about_the_largest(dtype, transposed):
    top = torch.finfo(dtype).max
    x = torch.zeros(6, 64, dtype=torch.float64)
    for i, f in enumerate((1.0, 0.9, 0.876, 0.874, 0.76, 0.5)):
        x[i, i], x[i, 32 + i] = f * top, -f * top
    x = x.to(dtype).to(DEV)
    want = x.double().cpu()
    for v in want.unique().tolist():
        if v:
            want[want == v] = math.copysign(_nearest(abs(v)), v)
    assert want.max() > top  # the largest ones pass the type's end
    assert torch.all((want - x.double().cpu()).abs() <= x.double().cpu().abs() / 4)
    q = M.mx_quantize_transposed(x.t().contiguous()) if transposed else M.mx_quantize(x)
    assert torch.equal(M.mx_restore(q, dtype).cpu(), want.to(dtype))
    # rows of one weight pick a value and scale it down into fp32's range: exact products
    w = torch.eye(64, device=DEV) * 2.0 ** -20
    y = M.mx_product(q, M.mx_quantize(w), dtype=torch.float32)
    assert torch.equal(y.cpu().double(), want * 2.0 ** -20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_about_the_smallest(dtype):
    """Blocks of the least exponent, -127: subnormals, held in steps of 2^-128 and taken by
    products as what they are."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    x = torch.zeros(8, 64, dtype=torch.float64)
    for i in range(8):
        x[i, :8] = grid.roll(i) * 2.0 ** -127
        x[i, 32:40] = -grid.roll(i) * 2.0 ** -127
    q = M.mx_quantize(x.to(dtype).to(DEV))
    assert torch.equal(x.to(dtype).double(), x) and not q.scales[0, :8, :2].any()
    assert torch.equal(M.mx_restore(q, dtype).cpu().double(), x)
    for up in (30, 100):
        w = torch.eye(64, device=DEV) * 2.0 ** up
        y = M.mx_product(q, M.mx_quantize(w), dtype=torch.float32)
        assert torch.equal(y.cpu().double(), x * 2.0 ** up)
    # below half the smallest step: zeros
    tiny = torch.full((1, 32), 2.0 ** -130).to(dtype).to(DEV)
    assert not M.mx_restore(M.mx_quantize(tiny), torch.float32).any()
