"""Router losses, expert counts and the router logits' gradient on the GPU against
plain 64-bit definitions.

Bounds: a softmax term is within 2e-6 (hardware exponential 2^-22, sum and quotient
a few 2^-24) for logits within 20 of the largest; sums over rows run in fp32 chains
of at most 16 rows, then 8 warps, then one term per chunk: 1e-5 relative covers
them.  A gradient entry is a difference of terms of that error: 1e-5 of the terms'
magnitudes.  Counts and tokens are whole numbers and equal.
"""
import math

import pytest
import torch

import nvfp4_token_routed_gb300 as M
import loss_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 1e-5
CB, CZ = 1e-2, 1e-3


def _batch(T, E, K, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, E, generator=g) + torch.randn(E, generator=g)).to(dtype)
    top = torch.topk(x.float(), K, dim=1)
    w = torch.softmax(top.values, 1)
    return x, top.indices.to(torch.int32), w, torch.randn(T, K, generator=g) * 1e-3


def _check(x, ids, w, dw, offsets=None, mask=None, grad=None, dlogits=None):
    c = [None if v is None else v.to(DEV) for v in (x, ids, w, dw, offsets, mask)]
    kw = dict(seq_offsets=c[4], token_mask=c[5])
    losses, counts, tokens = M.router_loss(c[0], c[1], CB, CZ, **kw)
    d = M.router_loss_grad(c[0], c[1], counts, tokens, CB, CZ, topk_w=c[2], d_topk_w=c[3],
                           loss_grad=None if grad is None else torch.tensor(grad, device=DEV),
                           dlogits=dlogits, **kw)
    want = R.router(x, ids, CB, CZ, offsets, mask, grad or (1.0, 1.0), w, dw)
    assert torch.equal(counts.cpu().long(), want[1])
    assert torch.equal(tokens.cpu().long(), want[2])
    assert torch.allclose(losses.cpu().double(), want[0], rtol=1e-5, atol=1e-12)
    R.check_grad(d, want[3], want[4], REL)
    return losses, counts, tokens, d


@pytest.mark.parametrize("E,K", [(1, 1), (8, 2), (33, 5), (64, 8), (100, 3), (256, 8), (384, 6),
                                 (1000, 32), (1024, 1)])
@pytest.mark.parametrize("T", [1, 2, 63, 300])
def test_losses_counts_and_gradient(T, E, K):
    _check(*_batch(T, E, K, T * 1000 + E))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_types_and_upstream_gradients(dtype):
    x, ids, w, dw = _batch(200, 96, 4, 3, dtype)
    _check(x, ids, w, dw, grad=(2.0, -0.5))
    _check(x, ids, None, None, grad=(0.0, 1.0))


@pytest.mark.parametrize("T,cuts", [(300, [0, 1, 1, 130, 131, 256, 300]), (5, [0, 0, 5, 5]),
                                    (700, [3, 127, 128, 129, 640]), (400, [0] * 40 + [400] * 9),
                                    (1000, list(range(0, 1001, 8)))])
def test_sequences_of_ragged_lengths(T, cuts):
    x, ids, w, dw = _batch(T, 40, 4, T)
    off = torch.tensor(cuts, dtype=torch.int32)
    g = torch.Generator().manual_seed(T)
    for mask in (None, torch.rand(T, generator=g) < 0.7, torch.zeros(T, dtype=torch.bool)):
        d = _check(x, ids, w, dw, offsets=off, mask=mask)[3]
        assert not d[:cuts[0]].any() and not d[cuts[-1]:].any()


def test_masked_rows_may_hold_anything_and_rows_without_a_finite_logit():
    x, ids, w, dw = _batch(150, 64, 8, 9)
    mask = torch.ones(150, dtype=torch.bool)
    mask[[0, 77, 149]] = False
    base = _check(x, ids, w, dw, mask=mask)
    bad = x.clone()
    bad[0], bad[77], bad[149] = math.nan, math.inf, -math.inf
    losses, counts, tokens = M.router_loss(bad.to(DEV), ids.to(DEV), CB, CZ,
                                           token_mask=mask.to(DEV))
    assert torch.equal(losses, base[0]) and torch.equal(counts, base[1])
    x[3] = -math.inf               # counts, but has no probabilities
    x[4, ::2] = -math.inf
    x[5, ::2] = torch.finfo(torch.float32).min
    x[6] = torch.finfo(torch.float32).min
    x[6, 1:] = -math.inf
    x6 = x.clone()
    x6[6] = 0.0                    # its squared log-sum-exp is not finite
    _check(x6, ids, w, dw, mask=mask.to(torch.uint8))
    x[7, 5] = math.nan
    losses, counts, _ = M.router_loss(x.to(DEV), ids.to(DEV), CB, CZ)
    assert torch.isnan(losses).any() and int(counts.sum()) == 150 * 8


def test_ids_empty_out_of_range_repeated_and_64_bit():
    x, ids, w, dw = _batch(140, 16, 4, 10)
    ids[0] = -1
    ids[1, 1:] = -1
    ids[2, 2] = ids[2, 1]
    base = _check(x, ids, w, dw)
    same = _check(x, ids.long(), w, dw)
    assert all(torch.equal(a, b) for a, b in zip(base, same))
    ws = M.router_loss_workspace(140, 16)
    M.router_loss(x.to(DEV), ids.to(DEV), CB, CZ, ws=ws)
    assert M.moe_nvfp4_read_status(ws) == 0
    for kind, value in ((torch.int32, 16), (torch.int32, -2), (torch.int64, (1 << 33) + 1)):
        far = ids.to(kind).clone()
        far[0] = value
        out = M.router_loss(x.to(DEV), far.to(DEV), CB, CZ, ws=ws)
        assert torch.equal(out[1], base[1]) and M.moe_nvfp4_read_status(ws) == 7
    M.router_loss(x.to(DEV), ids.to(DEV), CB, CZ, ws=ws)
    assert M.moe_nvfp4_read_status(ws) == 0


def test_strides_and_gradient_in_place():
    T, E, K = 130, 48, 4
    x, ids, w, dw = _batch(T, E, K, 11)
    store = torch.zeros(T, E + 5, device=DEV)
    view = store[:, 3:3 + E]
    view.copy_(x)
    losses, counts, tokens = M.router_loss(view, ids.to(DEV), CB, CZ)
    args = (ids.to(DEV), counts, tokens, CB, CZ)
    sc = dict(topk_w=w.to(DEV), d_topk_w=dw.to(DEV))
    plain = M.router_loss_grad(x.to(DEV), *args, **sc)
    out = M.router_loss_grad(view, *args, dlogits=view, **sc)
    assert torch.equal(out, plain)
    assert not store[:, :3].any() and not store[:, 3 + E:].any()


def test_same_bits_again_and_workspace_contents_do_not_matter():
    x, ids, w, dw = _batch(5000, 256, 8, 12)
    xc, ic = x.to(DEV), ids.to(DEV)
    off = torch.tensor([0, 1700, 1701, 4000, 5000], dtype=torch.int32, device=DEV)
    ws = M.router_loss_workspace(5000, 256, 4)
    first = M.router_loss(xc, ic, CB, CZ, seq_offsets=off, ws=ws)
    ws.fill_(0xFF)
    again = M.router_loss(xc, ic, CB, CZ, seq_offsets=off, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = M.router_loss(xc, ic, CB, CZ, seq_offsets=off, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))


def test_long_batches():
    """Against float64 sums on the GPU, for sizes past the row loops of the definitions."""
    for T, E, K in ((20000, 256, 8), (70001, 60, 3)):
        x, ids, _, _ = _batch(T, E, K, T)
        losses, counts, tokens = M.router_loss(x.to(DEV), ids.to(DEV), CB, CZ)
        c = torch.bincount(ids.reshape(-1).long(), minlength=E)
        assert torch.equal(counts.cpu()[0].long(), c) and tokens.tolist() == [T, T]
        p = torch.softmax(x.double(), 1).sum(0)
        bal = CB / T * (c.double() * E / (K * T) * p).sum()
        z = CZ / T * (torch.logsumexp(x.double(), 1) ** 2).sum()
        assert torch.allclose(losses.cpu().double(), torch.stack([bal, z]), rtol=1e-5)


def test_even_load_gives_the_coefficient():
    T, E, K = 64, 32, 1
    x = torch.zeros(T, E, device=DEV)
    ids = (torch.arange(T, device=DEV) % E).to(torch.int32).reshape(T, K)
    losses, counts, _ = M.router_loss(x, ids, 1.0, 1.0)
    assert (counts == T // E).all()
    assert abs(float(losses[0]) - 1.0) < 1e-6 and abs(float(losses[1]) - math.log(E) ** 2) < 1e-4


def test_gradient_against_differences():
    """The counts are constants: the 64-bit losses along random directions, with the
    counts of the unmoved batch."""
    T, E, K, h = 12, 20, 3, 1e-4
    x, ids, _, _ = _batch(T, E, K, 13)
    d = _check(x, ids, None, None)[3].cpu().double()
    mag = R.router(x, ids, CB, CZ)[4]
    g = torch.Generator().manual_seed(14)

    def value(v):
        return R.router(v, ids, CB, CZ)[0].sum()
    for _ in range(5):
        step = torch.randn(T, E, generator=g, dtype=torch.float64)
        diff = (value(x.double() + h * step) - value(x.double() - h * step)) / (2 * h)
        tol = 1e-4 * abs(float(diff)) + REL * float((mag * step.abs()).sum())
        assert abs(float((d * step).sum() - diff)) <= tol


def test_score_gradient_against_differences():
    """sum(dw * route_topk(x).scores) along random directions, while the choice stays."""
    T, E, K, h = 9, 16, 4, 1e-5
    x, ids, w, dw = _batch(T, E, K, 15)
    lg = x.to(DEV)
    rid, rw = M.route_topk(lg, K)
    _, counts, tokens = M.router_loss(lg, rid, 0.0, 0.0)
    d = M.router_loss_grad(lg, rid, counts, tokens, 0.0, 0.0, topk_w=rw, d_topk_w=dw.to(DEV))
    g = torch.Generator().manual_seed(16)

    def value(v):
        return (torch.softmax(v.gather(1, rid.cpu().long()), 1) * dw.double()).sum()
    for _ in range(5):
        step = torch.randn(T, E, generator=g, dtype=torch.float64)
        diff = (value(x.double() + h * step) - value(x.double() - h * step)) / (2 * h)
        tol = 1e-4 * abs(float(diff)) + REL * float((w.abs() * dw.abs()).sum()) * 10
        assert abs(float((d.cpu().double() * step).sum() - diff)) <= tol


def test_no_rows():
    x = torch.empty(0, 8, device=DEV)
    ids = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    losses, counts, tokens = M.router_loss(x, ids, CB, CZ)
    assert not losses.any() and not counts.any() and not tokens.any()
    assert M.router_loss_grad(x, ids, counts, tokens, CB, CZ).shape == (0, 8)


def test_refusals():
    x = torch.zeros(6, 8, device=DEV)
    ids = torch.zeros(6, 2, dtype=torch.int32, device=DEV)
    f = torch.zeros(6, 2, device=DEV)
    off = torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    losses, counts, tokens = M.router_loss(x, ids, CB)
    for call in (
            lambda: M.router_loss(x.cpu(), ids, CB), lambda: M.router_loss(x, ids.cpu(), CB),
            lambda: M.router_loss(x, ids[:3], CB), lambda: M.router_loss(x, ids.float(), CB),
            lambda: M.router_loss(x, ids, CB, seq_offsets=off.long()),
            lambda: M.router_loss(x, ids, CB, seq_offsets=off[:1]),
            lambda: M.router_loss(x, ids, CB, token_mask=torch.ones(6, device=DEV)),
            lambda: M.router_loss(x, ids, CB, counts=torch.zeros(8, dtype=torch.int32, device=DEV)),
            lambda: M.router_loss_grad(x, ids, counts[:, :4], tokens, CB),
            lambda: M.router_loss_grad(x, ids, counts, tokens, CB, topk_w=f[:3], d_topk_w=f)):
        with pytest.raises(ValueError):
            call()
    big = torch.zeros(2, 1025, device=DEV)
    for code, call in (
            (2, lambda: M.router_loss(big, ids[:2], CB)),
            (2, lambda: M.router_loss(x, torch.zeros(6, 9, dtype=torch.int32, device=DEV), CB)),
            (1, lambda: M.router_loss(x, ids[:, :0], CB)),
            (1, lambda: M.router_loss(x, ids, math.inf)),
            (4, lambda: M.router_loss(x, ids, CB, ws=torch.empty(256, dtype=torch.uint8,
                                                                 device=DEV))),
            (1, lambda: M.router_loss_grad(x, ids, counts, tokens, CB, topk_w=f))):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.code == code
