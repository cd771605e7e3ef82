"""Router losses where their arithmetic leaves fp32, against plain 64-bit definitions."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
CB = 1e-2


@pytest.mark.parametrize("T,E", [(5, 8), (300, 33), (5000, 64)])
def test_a_z_loss_switched_off_is_zero(T, E):
    """Rows whose squared log-sum-exp is beyond fp32 (every logit of the lowest value)."""
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T))
    x[T // 2] = torch.finfo(torch.float32).min
    ids = torch.zeros(T, 1, dtype=torch.int32)
    losses, counts, tokens = M.router_loss(x.to(DEV), ids.to(DEV), CB, 0.0)
    p = torch.softmax(x.double(), 1)[:, 0].sum()
    assert abs(float(losses[0]) - float(CB / T * E * p)) <= 1e-5 * float(CB / T * E * p)
    assert float(losses[1]) == 0.0
    d = M.router_loss_grad(x.to(DEV), ids.to(DEV), counts, tokens, CB, 0.0)
    assert torch.isfinite(d).all()
    x[0, 0] = float("nan")  # still reaches both
    assert torch.isnan(M.router_loss(x.to(DEV), ids.to(DEV), CB, 0.0)[0]).all()
