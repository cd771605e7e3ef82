"""Failure detection of the vocabulary losses: a role of one block that leaves (as when its
bounded wait runs out) ends in NaN for every row it leaves unfinished, whichever block and
role it was, in right results for all others, and in a context that goes on working."""
import time

import pytest
import torch

import nvfp4_token_routed_gb300 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
CONSUMERS, PRODUCER, GATHER, FINISH = range(4)


def _inputs(N, V):
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.randn(N, V, generator=g, device=DEV).to(torch.bfloat16)
    a = torch.randint(V, (N,), generator=g, device=DEV)
    a[6] = -1
    a[12] = -1  # a row left out, among those that get NaN
    lp = M.token_logp(z, a)
    return z, a, lp - 0.1, torch.ones(N, device=DEV)


@pytest.mark.parametrize("V,role,rank", [
    (80000, CONSUMERS, 1), (80000, CONSUMERS, 0), (80000, PRODUCER, 1), (80000, GATHER, 1),
    (80000, GATHER, 0), (80000, FINISH, 1), (30000, CONSUMERS, 0), (30000, GATHER, 0)])
def test_rows_left_unfinished_are_nan(V, role, rank):
    N, row = 4 * 9 + 3, 8
    z, a, old, adv = _inputs(N, V)
    want = M.policy_loss_grad(z, a, old, adv)
    torch.cuda.synchronize()
    t0 = time.time()
    loss, logp, d = M.moe_nvfp4_selftest_loss_timeout(z, a, old, adv, role, rank, row)
    torch.cuda.synchronize()
    assert time.time() - t0 < 20.0
    lost = torch.zeros(N, dtype=torch.bool, device=DEV)
    lost[row::4] = True
    assert torch.isnan(loss[lost]).all() and torch.isnan(logp[lost]).all(), (loss, logp)
    assert torch.equal(loss[~lost], want[0][~lost]) and torch.equal(logp[~lost], want[1][~lost])
    assert torch.equal(d[~lost], want[2][~lost])
    again = M.policy_loss_grad(z, a, old, adv)  # the context still works
    assert all(torch.equal(x, y) for x, y in zip(again, want))


def test_refusals():
    z, a, old, adv = _inputs(16, 80000)
    for code, call in ((1, (z, a, old, adv, 4, 0, 0)), (1, (z, a, old, adv, 0, 2, 0)),
                       (1, (z, a, old, adv, 0, 0, -1)), (2, (z[:, :8000], a, old, adv, 0, 0, 0)),
                       (2, (z.float(), a, old, adv, 0, 0, 0))):
        with pytest.raises(M.MoeError) as e:
            M.moe_nvfp4_selftest_loss_timeout(*call)
        assert e.value.code == code
