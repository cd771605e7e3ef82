"""A limit that is not 0 but that fp32 holds as 0 would switch the clamp off: refused."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M


def test_limits_that_fp32_rounds_to_zero():
    codes, scales = torch.zeros(4, 2, 32, dtype=torch.uint8), torch.zeros(4, 2, 1, dtype=torch.uint8)
    for limit in (1e-50, -1e-50, 2.0 ** -151):
        with pytest.raises(ValueError):
            M.Checkpoint(codes, scales, 8, torch.float32, "swiglu", limit)
    for limit in (0.0, -0.0, 2.0 ** -149, 1, float("inf")):
        assert M.Checkpoint(codes, scales, 8, torch.float32, "swiglu", limit).swiglu_limit == limit


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [False, True])
def test_calls_with_such_limits(keep):
    h = torch.full((3, 64), 2.0, device="cuda")
    M.expert_act(h, "swiglu", 0.0, keep)  # the library is there: compiled from here on
    with pytest.raises(ValueError):
        M.expert_act(h, "swiglu", 1e-50, keep)
    with pytest.raises(ValueError):
        M.MxExperts(torch.randn(2, 64, 32, device="cuda"), torch.randn(2, 32, 32, device="cuda"),
                    "swiglu", 1e-50)
    y = M.expert_act(h, "swiglu", 2.0 ** -100, keep)
    want = 2.0 ** -201  # L s(L) L, s(L) = 1/2: below fp32's range
    assert want < 2.0 ** -150 and torch.all((y[0] if keep else y) == 0.0)
