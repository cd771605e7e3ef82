"""Vocabulary losses where their arithmetic leaves the ordinary range, against plain
64-bit definitions.  Bounds as in test_gpu_token_loss.py: REL of the terms of a gradient,
1e-5 and 2^-20 of the magnitudes for a log-probability, tau^2 times that for a divergence.
"""
import math

import pytest
import torch

import nvfp4_token_routed_gb300 as M
import loss_refs as R
from test_gpu_token_loss import (DEV, REL, TYPES, _check_policy, _cuda, _policy_inputs,
                                 _run_policy)

pytestmark = pytest.mark.gpu
SHAPES = [37, 1000, 4096, 50001]


def _rows(V, dtype, fill, seed):
    """Rows with masked columns of one finite value; also the columns that may be chosen."""
    g = torch.Generator().manual_seed(seed)
    z = (2.0 * torch.randn(7, V, generator=g)).to(TYPES[dtype])
    keep = torch.ones(7, V, dtype=torch.bool)
    keep[0, [0, V - 1]] = False          # the first and last column
    keep[1, :3 * V // 4] = False         # what the first vectors hold
    keep[2] = False
    keep[2, V // 2] = True               # all but one
    keep[3] = False                      # all: uniform
    keep[4, ::2] = False
    keep[5, 1:V // 2] = False
    z[~keep] = fill
    z[6, V // 2:] = 0.5 * fill           # masked a second time, by half as much
    keep[6, V // 2:] = False
    pick = keep.clone()
    pick[3] = True
    ids = torch.multinomial(pick.float(), 4, replacement=True, generator=g)
    return z, ids


@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("dtype,fill,tau", [
    ("f32", -1e9, 1.0), ("f32", -1e10, 1.0), ("f32", -1e20, 0.7), ("f32", -1e30, 1.0),
    ("f32", "lowest", 5.0), ("f32", "lowest", 8.0), ("bf16", -1e9, 1.0), ("bf16", -1e10, 1.0),
    ("bf16", -1e20, 2.0), ("bf16", -1e30, 1.0), ("bf16", "lowest", 5.0),
    ("bf16", "lowest", 6.0), ("bf16", "lowest", 8.0), ("f16", "lowest", 0.5)])
def test_masks_of_any_finite_value(V, dtype, fill, tau):
    if fill == "lowest":
        fill = torch.finfo(TYPES[dtype]).min
    z, ids = _rows(V, dtype, fill, V)
    g = torch.Generator().manual_seed(V + 1)
    N = z.shape[0]
    store = torch.zeros(N, V + 2, dtype=z.dtype, device=DEV)
    for zc in (z.to(DEV), store[:, 1:1 + V].copy_(z)):  # rows on and off 16-byte boundaries
        t, w = torch.randn(N, 4, generator=g), torch.rand(N, generator=g) + 0.1
        ic, tc, wc = _cuda(ids, t, w)
        loss, d = M.distill_loss_grad(zc, ic, tc, wc, temperature=tau)
        want, dw, mag = R.distill(z, ids, t, None, w, tau)
        tol = tau * tau * (1e-5 + 2.0 ** -20 * 30)
        assert torch.all((loss.cpu().double() - want).abs() <= tol), (loss.cpu(), want)
        R.check_grad(d, dw, mag, REL)
        assert torch.equal(M.distill_loss(zc, ic, tc, temperature=tau), loss)
        a = ids[:, 0].contiguous()
        x = z.double() / tau
        lp = torch.log_softmax(x, 1).gather(1, a[:, None])[:, 0]
        old, adv = (lp + 0.5).float(), torch.randn(N, generator=g)
        out = _run_policy(z, a, old, adv, None, w, tau)
        _check_policy(out, z, a, old, adv, None, w, tau)
        got = M.token_logp(zc, a.to(DEV), temperature=tau).cpu().double()
        assert torch.all((got - lp).abs() <= 1e-5 + 2.0 ** -20 * (1.0 + lp.abs()))


@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("at", [1.0, 2.0 ** 21, 2.0 ** 22, 2.0 ** 23, 2.0 ** 26])
def test_logits_about_a_large_value(V, at):
    """Rows whose logits straddle the size at which exponents are taken another way: +-at in
    units of log2 e, less than 60 apart."""
    g = torch.Generator().manual_seed(V)
    step = max(0.25, at * 2.0 ** -23)
    n = int(30 / step)
    for sign in (1.0, -1.0):
        z = (sign * at / 1.4426950408889634
             + step * torch.randint(-n, n + 1, (4, V), generator=g).float())
        a = torch.randint(V, (4,), generator=g)
        x = z.double()
        lp = torch.log_softmax(x, 1).gather(1, a[:, None])[:, 0]
        old, adv, w = (lp + 0.5).float(), torch.randn(4, generator=g), torch.ones(4)
        _check_policy(_run_policy(z, a, old, adv, None, w, 1.0), z, a, old, adv, None, w, 1.0)


@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tau", [1.0, 3.0])
def test_tokens_of_the_lowest_value(V, dtype, tau):
    """A chosen token, or all of a teacher's, at the type's lowest logit: a finite
    log-probability of about that size, no gradient from the row's other tokens lost."""
    g = torch.Generator().manual_seed(V)
    lowest = torch.finfo(TYPES[dtype]).min
    z = torch.randn(3, V, generator=g).to(TYPES[dtype])
    z[:, [0, V // 2, V - 1]] = lowest
    z[2] = -math.inf               # nothing but a token of the lowest value: probability 1
    z[2, V // 2] = lowest
    a = torch.tensor([0, V - 1, V // 2])
    x = z.double() / tau
    lp = torch.log_softmax(x, 1).gather(1, a[:, None])[:, 0]
    got = M.token_logp(z.to(DEV), a.to(DEV), temperature=tau).cpu().double()
    assert torch.allclose(got, lp, rtol=1e-5, atol=2e-5), (got, lp)
    ids = torch.tensor([[0, V // 2], [V - 1, V - 1], [V // 2, V // 2]])
    t = torch.randn(3, 2, generator=g)
    # half the mass, so that the loss stays within fp32 (tau^2 Q (3.4e38 / tau))
    lse = torch.logsumexp(t / tau, 1) + math.log(8.0)
    loss, d = M.distill_loss_grad(*_cuda(z, ids, t), teacher_lse=lse.to(DEV), temperature=tau)
    want, dw, mag = R.distill(z, ids, t, lse, None, tau)
    assert torch.allclose(loss.cpu().double(), want, rtol=1e-5, atol=tau * tau * 4e-5), (loss, want)
    R.check_grad(d, dw, mag, REL)


@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zero_advantage_with_a_ratio_beyond_fp32(V, dtype):
    """A row without an advantage costs nothing, however far its policy has moved; a NaN
    in its logits still reaches it."""
    z = torch.randn(5, V, generator=torch.Generator().manual_seed(V)).to(TYPES[dtype])
    a = torch.zeros(5, dtype=torch.int64)
    lp = z.double()[:, 0] - torch.logsumexp(z.double(), 1)
    old, adv = (lp - 100.0).float(), torch.tensor([0.0, -0.0, 1.0, 0.0, 0.0])
    ref = (lp + 0.3).float()
    z[4, V - 1] = math.nan
    zc, ac, oc, vc, rc = _cuda(z, a, old, adv, ref)
    for r, beta in ((None, 0.0), (rc, 0.1)):
        loss, _, d = M.policy_loss_grad(zc, ac, oc, vc, ref_logp=r, clip_low=0.2, clip_high=0.28,
                                        kl_coef=beta)
        want, _, dw, mag = R.policy(z[:4], a[:4], old[:4], adv[:4], None if r is None else ref[:4],
                                    None, 0.2, 0.28, beta, 1.0)
        assert torch.all((loss[:4].cpu().double() - want).abs() <= 2e-5), loss
        R.check_grad(d[:4], dw, mag, 2 * REL)
        assert torch.isnan(loss[4]) and torch.isnan(d[4].float()).any()
        only = M.policy_loss(zc, ac, oc, vc, ref_logp=r, clip_low=0.2, clip_high=0.28, kl_coef=beta)
        assert torch.equal(only[0][:4], loss[:4])


@pytest.mark.parametrize("V", SHAPES)
def test_a_kl_term_switched_off_adds_nothing(V):
    """kl_coef 0 with a reference at hand: as without one, whatever the reference holds."""
    z = torch.randn(5, V, generator=torch.Generator().manual_seed(V))
    a = torch.zeros(5, dtype=torch.int64)
    z[0, 0] = -math.inf                   # a chosen token that is masked
    lp = z.double()[:, 0] - torch.logsumexp(z.double(), 1)
    old = torch.where(torch.isfinite(lp), lp, -3.0).float()
    ref = (lp + torch.tensor([0.0, 100.0, -1e30, math.inf, math.nan])).float()
    ref[0] = -3.0
    zc, ac, oc, rc = _cuda(z, a, old, ref)
    adv = torch.ones(5, device=DEV)
    plain = M.policy_loss_grad(zc, ac, oc, adv)
    off = M.policy_loss_grad(zc, ac, oc, adv, ref_logp=rc, kl_coef=0.0)
    assert torch.isfinite(plain[0]).all() and torch.isfinite(plain[2]).all()
    assert all(torch.equal(x, y) for x, y in zip(plain, off)), (plain, off)
    assert all(torch.equal(x, y) for x, y in zip(
        M.policy_loss(zc, ac, oc, adv, ref_logp=rc), M.policy_loss(zc, ac, oc, adv)))


@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("weight", [1.0, 2.0 ** -9])
def test_gradients_about_the_limit_of_the_folded_factor(V, dtype, weight):
    """16-bit gradients whose reference exponent is about 256 in size, on either side of it:
    temperature 0.1, logits about 17.75."""
    g = torch.Generator().manual_seed(V)
    z = 2.0 * torch.randn(6, V, generator=g)
    for i, top in enumerate((17.5, 17.75, 18.0)):
        z[i, torch.randint(V, (9,), generator=g)] = top
        z[i + 3] = -top + 0.125 * torch.randint(-3, 4, (V,), generator=g).float()
    z = z.to(TYPES[dtype])
    a = z.float().argmax(1)
    x = z.double() / 0.1
    lp = torch.log_softmax(x, 1).gather(1, a[:, None])[:, 0]
    old, adv = (lp + 0.5).float(), torch.randn(6, generator=g)
    w = torch.full((6,), weight)
    _check_policy(_run_policy(z, a, old, adv, None, w, 0.1), z, a, old, adv, None, w, 0.1)


@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_policy_loss_without_a_gradient(V, dtype):
    z = (2.0 * torch.randn(9, V, generator=torch.Generator().manual_seed(V))).to(TYPES[dtype])
    a, old, adv, ref, w = _policy_inputs(z, V, 0.8)
    loss, logp, _ = _run_policy(z, a, old, adv, ref, None, 0.8)
    _check_policy(_run_policy(z, a, old, adv, ref, w, 0.8), z, a, old, adv, ref, w, 0.8)
    zc, ac, oc, vc, rc = _cuda(z, a, old, adv, ref)
    only = M.policy_loss(zc, ac, oc, vc, ref_logp=rc, clip_low=0.2, clip_high=0.28, kl_coef=0.1,
                         temperature=0.8)
    assert torch.equal(only[0], loss) and torch.equal(only[1], logp)


@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_of_neighbouring_values_about_a_billion(V, dtype):
    """Rows of a few neighbouring values, +-2^28 .. 2^34 in units of log2 e: the largest share
    the row, as every other is 64 and more lower."""
    g = torch.Generator().manual_seed(V)
    bits = 23 if dtype == "f32" else 7
    for e in (28, 30, 31, 32, 34):
        for sign in (1.0, -1.0):
            mid = sign * 2.0 ** e / 1.4426950408889634
            ulp = 2.0 ** (math.floor(math.log2(abs(mid))) - bits)
            z = (round(mid / ulp) + torch.randint(-3, 4, (4, V), generator=g)).double() * ulp
            assert torch.equal(z.to(TYPES[dtype]).double(), z)
            z = z.to(TYPES[dtype])
            a = torch.cat([z[:2].float().argmax(1), torch.randint(V, (2,), generator=g)])
            lp = torch.log_softmax(z.double(), 1).gather(1, a[:, None])[:, 0]
            old = M.token_logp(z.to(DEV), a.to(DEV)).cpu()
            assert torch.all((old.double() - lp).abs() <= 1e-5 + 2.0 ** -20 * (1.0 + lp.abs()))
            # the ratio is 1: a gradient of probabilities alone, those of 2^-64 and less apart
            w = torch.full((4,), 0.5)
            d = _run_policy(z, a, old, torch.ones(4), None, w, 1.0)[2].cpu().double()
            p = torch.softmax(z.double(), 1)
            want = 0.5 * p
            want[torch.arange(4), a] -= 0.5
            assert torch.all((d - want).abs() <= R.ROUND[z.dtype][0] * want.abs() + REL + 2e-19)
