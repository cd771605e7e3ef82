"""Policy loss, token log-probability and distillation on the GPU against plain
64-bit definitions.

Bounds, from the arithmetic.  p_j = 2^((z_j - m) c) / s: the hardware exponential
is within 2 ulp (2^-22), the rounding of its argument x adds |x| ln 2 2^-23, at most
150 * 2^-23.5 < 1.3e-5 where p_j does not underflow, and s is a sum of positive fp32
terms, whose error stays below a few 2^-22 in practice and below 1.6e-5 for chains
of 256 terms in the worst case: REL = 3e-5 on every term of a gradient.  log s has
that as an absolute error, but its large terms have small |x|: 1e-5 absolute plus
2^-22 of the magnitudes involved for a log-probability; a KL divergence or a policy
loss carries it times its slope.
"""
import math

import pytest
import torch

import nvfp4_token_routed_gb300 as M
import loss_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 3e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = [1, 2, 7, 31, 255, 1000, 4096, 8191, 16384, 50001, 65528, 131072, 262144]


def _logits(N, V, dtype, seed, pad=0, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V + pad, generator=g) * scale
    hot = torch.randint(V, (N, 5), generator=g)
    z.scatter_(1, hot, 6.0 + 4.0 * torch.rand(N, 5, generator=g))
    return z.to(TYPES[dtype])


def _policy_inputs(z, seed, tau):
    g = torch.Generator().manual_seed(seed)
    N, V = z.shape
    a = torch.randint(V, (N,), generator=g)
    lp = (z.double() / tau).gather(1, a[:, None])[:, 0] - torch.logsumexp(z.double() / tau, 1)
    # well off the clipping edges at 1 - 0.2 and 1 + 0.28: which side a row is on is certain
    move = torch.tensor([-0.5, -0.1, 0.1, 0.5])[torch.randint(4, (N,), generator=g)]
    return (a, (lp - move).float(), torch.randn(N, generator=g),
            (lp + 0.3 * torch.randn(N, generator=g)).float(), torch.rand(N, generator=g) + 0.1)


def _teacher(z, k, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    t = z.float() + 0.5 * torch.randn(z.shape, generator=g)
    top = torch.topk(t, k, dim=1)
    return top.indices.to(torch.int32), top.values.to(dtype), t


def _cuda(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _loss_tol(want, slope=1.0):
    return slope * 1e-5 + 2.0 ** -20 * (1.0 + want.abs())


def _run_policy(z, a, old, adv, ref, w, tau, beta=0.1, **kw):
    zc, ac, oc, vc, rc, wc = _cuda(z, a, old, adv, ref, w)
    return M.policy_loss_grad(zc, ac, oc, vc, wc, ref_logp=rc, clip_low=0.2, clip_high=0.28,
                              kl_coef=beta if ref is not None else 0.0, temperature=tau, **kw)


def _check_policy(out, z, a, old, adv, ref, w, tau, beta=0.1):
    loss, logp, d, mag = R.policy(z, a, old, adv, ref, w, 0.2, 0.28, beta, tau)
    r = torch.exp((logp - old.double()).clamp(-30, 3))
    slope = r * adv.double().abs() + 1.0
    assert torch.all((out[1].cpu().double() - logp).abs() <= _loss_tol(logp)), "logp"
    assert torch.all((out[0].cpu().double() - loss).abs() <= _loss_tol(loss, slope)), "loss"
    # the softmax's error and the slope's, each within REL of its terms
    R.check_grad(out[2], d, mag, 2 * REL)


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_policy_matches_the_definition(V, dtype):
    N = 5 if V > 60000 else 9
    for tau, with_ref, pad in ((1.0, True, 0), (0.7, False, 3)):
        z = _logits(N, V, dtype, V + 1, pad)[:, :V]
        a, old, adv, ref, w = _policy_inputs(z, V + 2, tau)
        ref = ref if with_ref else None
        _check_policy(_run_policy(z, a, old, adv, ref, w, tau), z, a, old, adv, ref, w, tau)


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_distill_matches_the_definition(V, dtype):
    N = 5 if V > 60000 else 9
    for k, tau, full, tt, pad in ((min(V, 33), 1.0, False, torch.float32, 0),
                                  (min(V, 256), 2.0, True, torch.float32, 5),
                                  (1, 0.5, False, torch.bfloat16, 8)):
        z = _logits(N, V, dtype, V + 3, pad)[:, :V]
        ids, t, whole = _teacher(z, k, V + 4, tt)
        lse = torch.logsumexp(whole / tau, 1) if full else None
        w = torch.rand(N, generator=torch.Generator().manual_seed(V)) + 0.1
        zc, ic, tc, lc, wc = _cuda(z, ids, t, lse, w)
        loss, d = M.distill_loss_grad(zc, ic, tc, wc, teacher_lse=lc, temperature=tau)
        want, dw, mag = R.distill(z, ids, t, lse, w, tau)
        # the divergence is a sum of q (log q - log p); each log is off by up to 2^-22 |log|
        tol = tau * tau * (1e-5 + 2.0 ** -20 * 30)
        assert torch.all((loss.cpu().double() - want).abs() <= tol), (V, k)
        R.check_grad(d, dw, mag, REL)
        assert torch.equal(M.distill_loss(zc, ic, tc, teacher_lse=lc, temperature=tau), loss)


def test_logp_and_loss_only_calls_agree_with_the_gradient_call():
    for V in (1000, 50001, 131072):
        z = _logits(6, V, "bf16", V)
        a, old, adv, ref, w = _policy_inputs(z, 3, 1.0)
        out = _run_policy(z, a, old, adv, ref, w, 1.0)
        zc, ac, oc, vc, rc = _cuda(z, a, old, adv, ref)
        assert torch.equal(M.token_logp(zc, ac), out[1])
        loss, logp = M.policy_loss(zc, ac, oc, vc, ref_logp=rc, clip_low=0.2, clip_high=0.28,
                                   kl_coef=0.1)
        assert torch.equal(loss, out[0]) and torch.equal(logp, out[1])
        assert torch.equal(M.token_logp(zc, ac.to(torch.int32)), out[1])


@pytest.mark.parametrize("V", [700, 10000, 20000, 60000])
@pytest.mark.parametrize("k", [1, 33, 64, 256])
def test_many_rows(V, k):
    """Many rows a block, some left out at random: the calls with and without a gradient
    give the same, right losses, rows that start on 16 bytes the same when cut out of the batch,
    and every gradient row sums to 0."""
    N = 6000 if V < 30000 else 2500
    z = _logits(64, V, "bf16", V + k).to(DEV)
    pick = torch.randint(64, (N,), generator=torch.Generator().manual_seed(k)).to(DEV)
    ids, t, _ = _teacher(z.cpu(), k, 5)
    want = R.distill(z.cpu(), ids, t, None, None, 1.0)[0].to(DEV)[pick]
    z, ids, t = z[pick], ids.to(DEV)[pick], t.to(DEV)[pick]
    w = (torch.rand(N, generator=torch.Generator().manual_seed(k + 1)) < 0.7).float().to(DEV)
    loss = M.distill_loss(z, ids, t)
    assert torch.all((loss.double() - want).abs() <= 1e-5 + 2.0 ** -20 * 30)
    for _ in range(5):
        assert torch.equal(M.distill_loss(z, ids, t), loss)
    got, d = M.distill_loss_grad(z, ids, t, w)
    assert torch.equal(got, loss * w)
    assert not d[w == 0].any()
    # bf16 rounding of V entries, each at most 2^-8 of its size, of a row whose positive
    # entries sum to at most 1
    assert torch.all(d.double().sum(1).abs() <= 2.0 ** -7)
    if V % 8:
        return  # rows that do not start on 16 bytes are summed in an order of their own
    rows = torch.tensor([0, 1, 151, 152, 999, N - 1], device=DEV)
    assert torch.equal(M.distill_loss(z[rows], ids[rows], t[rows]), loss[rows])
    same = M.distill_loss_grad(z[rows], ids[rows], t[rows], w[rows])
    assert torch.equal(same[1], d[rows])
    a = ids[:, 0].clone()
    a[::7] = -1
    lp = M.token_logp(z, a)
    zero = torch.zeros(N, device=DEV)
    out = M.policy_loss_grad(z, a, zero - 1.0, zero + 1.0, w)
    assert torch.equal(out[1], lp * w) and torch.equal(M.token_logp(z[rows], a[rows]), lp[rows])
    assert not out[2][(w == 0) | (a < 0)].any()


@pytest.mark.parametrize("V", [49152, 49153, 98304, 98311, 196608, 196616])
def test_many_rows_of_full_parts(V):
    """Rows whose parts are the longest that one, two and four blocks take, and a little more."""
    test_many_rows(V, 33)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [37, 1000, 50001])
def test_masked_vocabulary_entries(V, dtype):
    N = 8
    z = _logits(N, V, dtype, V)
    lowest = torch.finfo(TYPES[dtype]).min
    z[0, ::2] = -math.inf
    z[1, ::2] = lowest
    z[2, :] = lowest               # all equal: uniform
    z[3, :] = -math.inf            # no finite logit: left out
    z[4, :] = -math.inf
    z[4, V // 2] = 1.5             # one token left: probability 1
    z[5, 1:] = lowest
    ids, t, _ = _teacher(torch.randn(N, V, generator=torch.Generator().manual_seed(1)), 4, 2)
    ids[0] = torch.tensor([1, 3, 5, 7])
    ids[1] = torch.tensor([0, 1, 3, 5])  # one of the lowest logits
    ids[4] = V // 2
    ids[5] = 0
    w = torch.ones(N)
    zc, ic, tc, wc = _cuda(z, ids, t, w)
    loss, d = M.distill_loss_grad(zc, ic, tc, wc)
    want, dw, mag = R.distill(z, ids, t, None, w, 1.0)
    big = want.abs() > 1e30  # the divergence from a token of the lowest logit
    tol = 1e-5 + 2.0 ** -19 * 30 + 2.0 ** -20 * want.abs()
    assert torch.all(((loss.cpu().double() - want).abs() <= tol)[~big])
    assert torch.allclose(loss.cpu().double()[big], want[big], rtol=1e-5)
    R.check_grad(d, dw, mag, REL)
    assert float(loss[3]) == 0.0 and not d[3].any()
    a = torch.full((N,), 1)
    a[4], a[5] = V // 2, 0
    old, adv = torch.full((N,), -1.0), torch.tensor([1.0, -1.0] * 4)
    lp = M.token_logp(zc, a.to(DEV)).cpu()
    assert float(lp[3]) == 0.0 and float(lp[4]) == 0.0 and float(lp[5]) == 0.0
    assert abs(float(lp[2]) + math.log(V)) < 1e-5
    out = _run_policy(z, a, old, adv, None, w, 1.0)
    assert not out[2][3].any() and torch.isfinite(out[2].float()).all()


def test_teacher_probability_on_a_masked_token_is_an_infinite_loss_with_a_finite_gradient():
    z = torch.zeros(1, 64)
    z[0, 5] = -math.inf
    ids = torch.tensor([[5, 6]], dtype=torch.int32)
    t = torch.tensor([[1.0, 0.0]])
    loss, d = M.distill_loss_grad(z.to(DEV), ids.to(DEV), t.to(DEV))
    assert float(loss) == math.inf and torch.isfinite(d).all()
    _, want, mag = R.distill(z, ids, t, None, None, 1.0)
    R.check_grad(d, want, mag, REL)


@pytest.mark.parametrize("V", [100, 40001, 131072])
def test_nan_and_inf_stay_in_their_rows(V):
    N = 6
    z = _logits(N, V, "f32", 5)
    a, old, adv, ref, w = _policy_inputs(z, 6, 1.0)
    ids, t, _ = _teacher(z, 4, 7)
    bad = z.clone()
    bad[1, V - 1] = math.nan
    bad[3, 0] = math.inf
    bad[4, V // 3] = math.nan
    w[4] = 0.0  # a row left out may hold anything
    a2 = a.clone()
    a2[3] = -1
    out = _run_policy(bad, a2, old, adv, ref, w, 1.0)
    ok = _run_policy(z, a, old, adv, ref, w, 1.0)
    for i in (0, 2, 5):
        assert torch.equal(out[2][i], ok[2][i]) and torch.equal(out[0][i], ok[0][i])
    assert torch.isnan(out[0][1]) and torch.isnan(out[1][1]) and torch.isnan(out[2][1]).any()
    for i in (3, 4):
        assert float(out[0][i]) == 0.0 and float(out[1][i]) == 0.0 and not out[2][i].any()
    loss, d = M.distill_loss_grad(*_cuda(bad, ids, t, w))
    assert torch.isnan(loss[1]) and torch.isnan(loss[3]) and float(loss[4]) == 0.0
    assert torch.isnan(d[1]).any() and torch.isnan(d[3]).any() and not d[4].any()
    assert torch.isfinite(d[[0, 2, 5]]).all()


def test_teacher_slots_empty_repeated_out_of_range_and_64_bit():
    V, N = 5000, 6
    z = _logits(N, V, "f32", 8)
    ids, t, _ = _teacher(z, 8, 9)
    ids[0, 3:] = -1
    ids[1] = -1                          # no teacher: left out
    ids[2, 4:] = ids[2, 0]               # one token in five slots
    ids[3, ::2] = torch.tensor([V, V + 7, 2 ** 31 - 1, -5], dtype=torch.int32)
    t[4] = -math.inf                     # no mass: left out
    t[5, 2] = -math.inf
    want, dw, mag = R.distill(z, ids, t, None, None, 1.0)
    for kind in (torch.int32, torch.int64):
        loss, d = M.distill_loss_grad(*_cuda(z, ids.to(kind), t))
        assert torch.all((loss.cpu().double() - want).abs() <= 1e-5 + 2.0 ** -20 * 30)
        R.check_grad(d, dw, mag, REL)
        assert float(loss[1]) == 0.0 and not d[1].any() and not d[4].any()
    far = ids.to(torch.int64)
    far[0, 3:] = (1 << 33) + 5           # would be token 5 in 32 bits
    loss2, d2 = M.distill_loss_grad(*_cuda(z, far, t))
    assert torch.equal(loss2, loss) and torch.equal(d2, d)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,pad,shift", [(999, 4, 1), (4096, 9, 3), (50000, 8, 8), (70001, 1, 0)])
def test_strided_and_unaligned_rows_and_gradients(V, pad, shift, dtype):
    N = 5
    store = _logits(N, V + pad, dtype, V).to(DEV)
    zc = store[:, shift:shift + V]
    z = zc.cpu()
    a, old, adv, ref, w = _policy_inputs(z, 1, 1.0)
    ac, oc, vc, rc, wc = _cuda(a, old, adv, ref, w)
    kw = dict(ref_logp=rc, clip_low=0.2, clip_high=0.28, kl_coef=0.1)
    for gpad, gshift in ((0, 0), (7, 2)):
        gs = torch.full((N, V + gpad), 77.0, dtype=store.dtype, device=DEV)
        view = gs[:, gshift:gshift + V]
        out = M.policy_loss_grad(zc, ac, oc, vc, wc, dlogits=view, **kw)
        assert out[2].data_ptr() == view.data_ptr()
        _check_policy(out, z, a, old, adv, ref, w, 1.0)
        rest = torch.ones(V + gpad, dtype=torch.bool)
        rest[gshift:gshift + V] = False
        assert (gs[:, rest.to(DEV)] == 77.0).all()  # nothing beside the rows is written
    # in place: the gradient takes the logits' storage
    before = store.clone()
    out = M.policy_loss_grad(zc, ac, oc, vc, wc, dlogits=zc, **kw)
    _check_policy(out, z, a, old, adv, ref, w, 1.0)
    zc.copy_(z)
    assert torch.equal(store, before)


def test_distill_in_place():
    V, N = 65536, 40
    z = _logits(N, V, "bf16", 3).to(DEV)
    ids, t, _ = _teacher(z.cpu(), 50, 4)
    ic, tc = _cuda(ids, t)
    loss, d = M.distill_loss_grad(z, ic, tc)
    loss2, d2 = M.distill_loss_grad(z, ic, tc, dlogits=z)
    assert d2.data_ptr() == z.data_ptr()
    assert torch.equal(loss, loss2) and torch.equal(d, d2)


@pytest.mark.parametrize("V", [512, 32000, 151936])
def test_rows_do_not_depend_on_the_batch(V):
    N = 300
    z = _logits(N, V, "bf16", V).to(DEV)
    a, old, adv, ref, w = [x.to(DEV) for x in _policy_inputs(z.cpu(), 1, 1.0)]
    kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.1)
    full = M.policy_loss_grad(z, a, old, adv, w, ref_logp=ref, **kw)
    again = M.policy_loss_grad(z, a, old, adv, w, ref_logp=ref, **kw)
    assert all(torch.equal(x, y) for x, y in zip(full, again))
    sel = torch.randperm(N, generator=torch.Generator().manual_seed(1))[:7].to(DEV)
    part = M.policy_loss_grad(z[sel], a[sel], old[sel], adv[sel], w[sel], ref_logp=ref[sel], **kw)
    assert all(torch.equal(x[sel], y) for x, y in zip(full, part))


def test_largest_rows_many_to_a_cluster():
    """fp32 rows of 2^18 logits: a block's part is more than half its ring."""
    V, N = 262144, 70
    z = _logits(8, V, "f32", 2).to(DEV)
    pick = torch.randint(8, (N,), generator=torch.Generator().manual_seed(3)).to(DEV)
    a, old, adv, ref, w = _policy_inputs(z.cpu(), 4, 1.0)
    one = _run_policy(z.cpu(), a, old, adv, ref, w, 1.0)
    _check_policy(one, z.cpu(), a, old, adv, ref, w, 1.0)
    p = pick.cpu()
    many = _run_policy(z[pick].cpu(), a[p], old[p], adv[p], ref[p], w[p], 1.0)
    assert all(torch.equal(x, y[pick]) for x, y in zip(many, one))
    assert torch.equal(M.token_logp(z[pick], a.to(DEV)[pick]), many[1])


def test_offsets_beyond_32_bits():
    V, N = 262144, 8600  # 2.25e9 logits: elements and bytes pass 2^31
    z = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)
    rows = [0, 8191, 8192, N - 1]
    z.zero_()
    z[rows] = _logits(4, V, "bf16", 1).to(DEV)
    a = torch.randint(V, (N,), device=DEV)
    lp = M.token_logp(z, a)
    assert torch.equal(lp[rows], M.token_logp(z[rows], a[rows]))
    w = torch.zeros(N, device=DEV)
    w[rows] = 1.0
    ones = torch.ones(N, device=DEV)
    small = M.policy_loss_grad(z[rows], a[rows], lp[rows], ones[:4])
    out = M.policy_loss_grad(z, a, lp, ones, w, dlogits=z)
    assert torch.equal(out[2][rows], small[2]) and not out[2][1].any() and not out[2][N - 2].any()


def test_clip_sides_and_edges():
    z = torch.zeros(8, 2, device=DEV)  # logp = -log 2
    lp = M.token_logp(z, torch.zeros(8, dtype=torch.int64, device=DEV))
    ratio = torch.tensor([0.5, 0.79, 1.0, 1.2, 1.29, 2.0, 0.5, 2.0], device=DEV)
    adv = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 1.0, -1.0, -1.0], device=DEV)
    loss, _, d = M.policy_loss_grad(z, torch.zeros(8, dtype=torch.int64, device=DEV),
                                    lp - torch.log(ratio), adv, clip_low=0.2, clip_high=0.28)
    want = torch.tensor([-0.5, -0.79, -1.0, -1.2, -1.28, -1.28, 0.8, 2.0], device=DEV)
    assert torch.allclose(loss, want, atol=1e-6)
    grad = torch.tensor([-0.25, -0.395, -0.5, -0.6, 0.0, 0.0, 0.0, 1.0], device=DEV)
    assert torch.allclose(d[:, 0], grad, atol=1e-6) and torch.allclose(d[:, 1], -grad, atol=1e-6)


@pytest.mark.parametrize("op", ["policy", "distill"])
def test_gradient_against_differences(op):
    """<grad, direction> against the central difference of the 64-bit loss: its error is
    h^2 times the third derivative (1e-6 here) plus rounding 1e-16 / h."""
    N, V, h = 4, 400, 1e-4
    z = _logits(N, V, "f32", 21)
    g = torch.Generator().manual_seed(22)
    w = torch.rand(N, generator=g) + 0.5
    if op == "policy":
        a, old, adv, ref, _ = _policy_inputs(z, 23, 1.3)
        grad = _run_policy(z, a, old, adv, ref, w, 1.3)[2]

        def value(x):
            return R.policy(x, a, old, adv, ref, w, 0.2, 0.28, 0.1, 1.3)[0]
    else:
        ids, t, whole = _teacher(z, 20, 24)
        lse = torch.logsumexp(whole / 1.3, 1)
        grad = M.distill_loss_grad(*_cuda(z, ids, t, w), teacher_lse=lse.to(DEV),
                                   temperature=1.3)[1]

        def value(x):
            return R.distill(x, ids, t, lse, w, 1.3)[0]
    for _ in range(5):
        step = torch.randn(N, V, generator=g, dtype=torch.float64)
        diff = (value(z.double() + h * step) - value(z.double() - h * step)) / (2 * h)
        along = (grad.cpu().double() * step).sum(1)
        assert torch.allclose(along, diff * w.double(), rtol=1e-4, atol=1e-4)


def test_another_stream_and_graph_replay():
    V, N = 32768, 64
    z = _logits(N, V, "bf16", 1).to(DEV)
    ids, t, _ = _teacher(z.cpu(), 32, 2)
    ic, tc = _cuda(ids, t)
    want = M.distill_loss_grad(z, ic, tc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = M.distill_loss_grad(z, ic, tc, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    torch.cuda.synchronize()
    loss, d = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.distill_loss_grad(z, ic, tc, row_loss=loss, dlogits=d)
    z.add_(torch.randn(N, V, device=DEV).to(z.dtype))
    graph.replay()
    torch.cuda.synchronize()
    fresh = M.distill_loss_grad(z, ic, tc)
    assert torch.equal(loss, fresh[0]) and torch.equal(d, fresh[1])


def test_no_rows():
    z = torch.empty(0, 100, device=DEV)
    a = torch.empty(0, dtype=torch.int32, device=DEV)
    f = torch.empty(0, device=DEV)
    assert M.token_logp(z, a).shape == (0,)
    assert M.policy_loss_grad(z, a, f, f)[2].shape == (0, 100)
    ids, t = torch.empty(0, 3, dtype=torch.int32, device=DEV), torch.empty(0, 3, device=DEV)
    assert M.distill_loss_grad(z, ids, t)[1].shape == (0, 100)


def test_refusals():
    z = torch.zeros(4, 100, device=DEV)
    a = torch.zeros(4, dtype=torch.int32, device=DEV)
    f = torch.zeros(4, device=DEV)
    ids, t = torch.zeros(4, 3, dtype=torch.int32, device=DEV), torch.zeros(4, 3, device=DEV)
    for call in (
            lambda: M.token_logp(z.cpu(), a), lambda: M.token_logp(z, a.cpu()),
            lambda: M.token_logp(z.t(), a), lambda: M.token_logp(z.double(), a),
            lambda: M.token_logp(z, a.float()), lambda: M.token_logp(z, a[:3]),
            lambda: M.token_logp(z[:1].expand(4, 100), a),
            lambda: M.token_logp(z, torch.zeros(8, dtype=torch.int32, device=DEV)[::2]),
            lambda: M.policy_loss(z, a, f.double(), f),
            lambda: M.policy_loss_grad(z, a, f, f, row_weight=f[:2]),
            lambda: M.policy_loss_grad(z, a, f, f, dlogits=torch.zeros(4, 99, device=DEV)),
            lambda: M.policy_loss_grad(z, a, f, f, dlogits=z.bfloat16()),
            lambda: M.distill_loss(z, ids, t[:, :2]), lambda: M.distill_loss(z, ids[:2], t[:2]),
            lambda: M.distill_loss(z, ids, t, teacher_lse=f[:2])):
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros(1, (1 << 18) + 1, device=DEV)
    many = torch.zeros(4, 257, dtype=torch.int32, device=DEV)
    for code, call in (
            (2, lambda: M.token_logp(wide, a[:1])),
            (1, lambda: M.token_logp(z, a, temperature=0.0)),
            (1, lambda: M.token_logp(z, a, temperature=math.nan)),
            (1, lambda: M.policy_loss(z, a, f, f, kl_coef=0.1)),
            (1, lambda: M.policy_loss(z, a, f, f, clip_low=1.5)),
            (1, lambda: M.policy_loss(z, a, f, f, clip_high=-0.1)),
            (1, lambda: M.distill_loss(z, ids[:, :0], t[:, :0])),
            (2, lambda: M.distill_loss(z, many, many.float()))):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.code == code
