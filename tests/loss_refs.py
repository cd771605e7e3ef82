"""Plain 64-bit definitions of the training objectives, row by row, for the tests.

Inputs are CPU tensors; every function returns float64 tensors.  `soft` and
`patch` are the magnitudes whose difference a gradient entry is: the kernels'
relative errors act on those, so the tests scale their bounds by them.
"""
import math

import torch

D = torch.float64


def _dist(z, tau):
    """(softmax, log-softmax) of one row over tau, or None for a row without a finite logit."""
    x = z.to(D) / tau
    m = x.max()
    if m == -math.inf:
        return None
    e = torch.exp(x - m)
    s = e.sum()
    return e / s, x - m - torch.log(s)


def policy(z, actions, old, adv, ref, weight, lo, hi, beta, tau):
    """(loss, logp, dlogits, scale) of the clipped policy loss; old None: logp only."""
    N, V = z.shape
    loss, logp = torch.zeros(N, dtype=D), torch.zeros(N, dtype=D)
    d, mag = torch.zeros(N, V, dtype=D), torch.zeros(N, V, dtype=D)
    for i in range(N):
        a = int(actions[i])
        w = 1.0 if weight is None else float(weight[i])
        if not 0 <= a < V or w == 0.0:
            continue
        row = _dist(z[i], tau)
        if row is None:
            continue
        p, lsm = row
        lp = float(lsm[a])
        logp[i] = lp
        if old is None:
            continue
        A, move = float(adv[i]), lp - float(old[i])
        r = math.exp(move) if move == move else math.nan
        c = min(max(r, 1.0 - lo), 1.0 + hi) if r == r else math.nan
        clipped = c * A < r * A
        value = -(c * A if clipped else r * A)
        g = 0.0 if clipped else -r * A
        terms = abs(g)  # the slope may be a difference of larger terms
        if ref is not None:
            x = float(ref[i]) - lp
            value += beta * (math.expm1(x) - x if x == x else math.nan)
            g -= beta * (math.expm1(x) if x == x else math.nan)
            terms += abs(beta) * (1.0 + (math.exp(x) if x == x else math.nan))
        loss[i] = value
        if g != 0.0:
            d[i] = -(w * g / tau) * p
            mag[i] = abs(w) * terms / tau * p
            d[i, a] += w * g / tau
            mag[i, a] += abs(w) * terms / tau
    return loss, logp, d, mag


def distill(z, ids, t, lse, weight, tau):
    """(loss, dlogits, scale) of the KL divergence to a teacher's top logits."""
    N, V = z.shape
    loss = torch.zeros(N, dtype=D)
    d, mag = torch.zeros(N, V, dtype=D), torch.zeros(N, V, dtype=D)
    for i in range(N):
        w = 1.0 if weight is None else float(weight[i])
        if w == 0.0:
            continue
        ok = (ids[i] >= 0) & (ids[i] < V)
        at = ids[i][ok].long()
        x = t[i][ok].to(D) / tau
        if not at.numel() or x.max() == -math.inf:
            continue
        lq = x - (torch.logsumexp(x, 0) if lse is None else lse[i].to(D))
        q = torch.exp(lq)
        row = _dist(z[i], tau)
        if row is None or float(q.sum()) == 0.0:
            continue
        p, lsm = row
        has = q != 0
        loss[i] = tau * tau * (q[has] * (lq[has] - lsm[at][has])).sum()
        Q = q.sum()
        pick = torch.zeros(V, dtype=D).index_add_(0, at, q)
        d[i] = w * tau * (Q * p - pick)
        mag[i] = abs(w) * tau * (Q * p + pick)
    return loss, d, mag


def router(x, ids, cb, cz, offsets=None, mask=None, grad=(1.0, 1.0), w=None, dw=None):
    """(losses, counts, tokens, dlogits, scale) of the router objectives."""
    T, E = x.shape
    K = ids.shape[1]
    cuts = [0, T] if offsets is None else [int(o) for o in offsets]
    S = len(cuts) - 1
    counts = torch.zeros(S, E, dtype=torch.int64)
    tokens = torch.zeros(S + 1, dtype=torch.int64)
    p, lse = torch.zeros(T, E, dtype=D), torch.zeros(T, dtype=D)
    seq = [-1] * T
    for s in range(S):
        for t in range(cuts[s], cuts[s + 1]):
            if mask is not None and not bool(mask[t]):
                continue
            seq[t] = s
            tokens[s] += 1
            row = _dist(x[t], 1.0)
            if row is not None:
                p[t] = row[0]
                lse[t] = torch.logsumexp(x[t].to(D), 0)
            for k in range(K):
                if 0 <= int(ids[t, k]) < E:
                    counts[s, int(ids[t, k])] += 1
    n = int(tokens.sum())
    tokens[S] = n
    d, mag = torch.zeros(T, E, dtype=D), torch.zeros(T, E, dtype=D)
    bal = z = torch.zeros((), dtype=D)
    for t in range(T):
        s = seq[t]
        if s < 0:
            continue
        f = counts[s].to(D) * E / (K * int(tokens[s]))
        dot = (f * p[t]).sum()
        bal = bal + cb / n * dot
        z = z + cz / n * lse[t] ** 2
        a, b = grad[0] * cb / n, grad[1] * 2 * cz / n * lse[t]
        d[t] = p[t] * (a * (f - dot) + b)
        mag[t] = p[t] * (abs(a) * (f + dot) + abs(b))
        if w is not None:
            ok = [k for k in range(K) if 0 <= int(ids[t, k]) < E]
            mean = sum(float(w[t, k]) * float(dw[t, k]) for k in ok)
            amean = sum(abs(float(w[t, k]) * float(dw[t, k])) for k in ok)
            for k in ok:
                d[t, int(ids[t, k])] += float(w[t, k]) * (float(dw[t, k]) - mean)
                mag[t, int(ids[t, k])] += float(w[t, k]) * (abs(float(dw[t, k])) + amean)
    return torch.stack([bal, z]), counts, tokens, d, mag


# Unit roundoff and smallest useful step of the gradient types.
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -126), torch.bfloat16: (2.0 ** -8, 2.0 ** -126),
         torch.float16: (2.0 ** -11, 2.0 ** -25)}


def check_grad(got, want, scale, rel):
    """|got - want| <= rounding of the type + rel * scale, elementwise; NaN where want is."""
    u, step = ROUND[got.dtype]
    g = got.detach().cpu().to(D)
    assert torch.equal(torch.isnan(g), torch.isnan(want))
    bound = u * want.abs() + (rel * scale) * (1 + u) + step
    bad = ((g - want).abs() > bound) & ~torch.isnan(want)
    assert not bad.any(), (int(bad.sum()), float(((g - want).abs() / bound)[bad].max()))
