"""Cases for the training-side operators around the routed expert layer, their
plain forms and their definitions in 64 bits.

Three groups, each with its gradient:
  router   balance loss, z loss and per-expert counts of the router logits, and
           the logits' gradient (with the routing scores' gradient folded in)
  distill  KL divergence to a teacher's top logits over the vocabulary
  policy   clipped policy loss with a KL term over the vocabulary, and the plain
           log-probability of chosen tokens ("logp")

`run` takes the framework's kernels where `own` is true, else elementary torch
operations in fp32, rounded once at the end.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MAX_ELEMS = 1 << 30  # logits of the largest vocabulary case

CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05
BALANCE_COEF, Z_COEF = 1e-2, 1e-3


# ------------------------------------------------------------------ cases

def _router(name, op, T, E, K, S=1, mask=False, dtype="f32"):
    c = {"op": op, "T": T, "E": E, "K": K, "S": S, "mask": mask, "dtype": dtype}
    return dict(c, name=name) if name else c


def _distill(name, op, N, V, k, tau, dtype="bf16", pad=0, banned=0.0, full=False):
    c = {"op": op, "N": N, "V": V, "k": k, "tau": tau, "dtype": dtype, "pad": pad,
         "banned": banned, "full": full}
    return dict(c, name=name) if name else c


def _policy(name, op, N, V, tau=1.0, dtype="bf16", pad=0, ref=True):
    c = {"op": op, "N": N, "V": V, "tau": tau, "dtype": dtype, "pad": pad, "ref": ref}
    return dict(c, name=name) if name else c


def listed():
    return [
        # expert load and router losses of a decode-sized batch, once per step and layer
        _router("router_loss_T64_E256", "router_loss", 64, 256, 8),
        # a small fine-tuning batch: losses, then the logits' gradient
        _router("router_step_T512_E64", "router_step", 512, 64, 8),
        # a prefill-sized training batch of the 384-expert layer
        _router("router_step_T4096_E384", "router_step", 4096, 384, 6),
        # packed sequences of ragged lengths, padding tokens masked, 16-bit logits
        _router("router_step_packed_T65536", "router_step", 65536, 256, 8, S=61, mask=True,
                dtype="bf16"),
        # held-out distillation loss of a short sequence
        _distill("distill_loss_N37_V32768", "distill_loss", 37, 32768, 32, 1.0),
        # distillation with rows of an odd vocabulary: no row but the first is aligned
        _distill("distill_grad_N1531_V100003", "distill_grad", 1531, 100003, 50, 1.5),
        # tokens ruled out by a mask (-inf) in student and teacher, fp32 logits, the
        # teacher's probabilities over its whole vocabulary
        _distill("distill_grad_f32_banned", "distill_grad", 2048, 65536, 64, 2.0, dtype="f32",
                 banned=0.3, full=True),
        # a full distillation batch: two sequences of 4096 tokens
        _distill("distill_grad_N8192_V131072", "distill_grad", 8192, 131072, 64, 1.0),
        # log-probabilities of the tokens that one decode step has chosen
        _policy("logp_N8_V131072", "logp", 8, 131072),
        # policy loss without a gradient over a scored batch
        _policy("policy_loss_N12000_V32000", "policy_loss", 12000, 32000, dtype="f16"),
        # a policy step on fp32 logits, without a reference policy
        _policy("policy_grad_f32_N1024_V50001", "policy_grad", 1024, 50001, dtype="f32",
                ref=False),
        # a policy step whose vocabulary is a slice of a padded head's output
        _policy("policy_grad_N6000_V151000", "policy_grad", 6000, 151000, tau=0.8, pad=72),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    group = rng.choice(["router", "distill", "distill", "policy", "policy"])
    if group == "router":
        E = rng.choice([8, 16, 33, 60, 64, 96, 128, 160, 256, 384, 512, 1000])
        K = rng.choice([k for k in (1, 2, 3, 4, 6, 8, 8, 10) if k <= E])
        T = _log_int(rng, 1, 65536)
        S = 1 if rng.random() < 0.5 else _log_int(rng, 1, min(T, 300))
        return _router(None, rng.choice(["router_loss", "router_step", "router_step"]), T, E, K, S,
                       rng.random() < 0.4, rng.choice(["f32", "f32", "bf16", "f16"]))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    V = _log_int(rng, 500, 262144)
    if rng.random() < 0.4:
        V = max(512, V // 128 * 128)
    most = MAX_ELEMS // (2 if dtype == "f32" else 1)
    N = _log_int(rng, 1, max(1, min(16384, most // V)))
    pad = rng.choice([0, 0, rng.randint(1, 200)])
    if group == "distill":
        return _distill(None, rng.choice(["distill_loss", "distill_grad", "distill_grad"]), N, V,
                        _log_int(rng, 1, 256), rng.choice([1.0, 1.0, 2.0, rng.uniform(0.5, 4.0)]),
                        dtype, pad, rng.choice([0.0, 0.0, 0.5]), rng.random() < 0.4)
    return _policy(None, rng.choice(["logp", "policy_loss", "policy_grad", "policy_grad"]), N, V,
                   rng.choice([1.0, 1.0, rng.uniform(0.6, 1.3)]), dtype, pad, rng.random() < 0.6)


# ------------------------------------------------------------------ inputs

def _chunk(V):
    return max(1, (1 << 26) // V)


def _vocab_logits(case, g):
    """Logits [N, V], a view of rows of V + pad values: a bell of small logits and
    sixteen tokens a row that stand out, as a language model's."""
    N, V, pad = case["N"], case["V"], case["pad"]
    store = torch.empty(N, V + pad, dtype=DTYPE[case["dtype"]], device="cuda")
    for r in range(0, N, _chunk(V)):
        n = min(_chunk(V), N - r)
        z = torch.randn(n, V + pad, generator=g, device="cuda") * 2.0
        at = torch.randint(V, (n, 16), generator=g, device="cuda")
        z.scatter_add_(1, at, 2.0 + 10.0 * torch.rand(n, 16, generator=g, device="cuda"))
        store[r:r + n] = z.to(store.dtype)
    return store[:, :V]


def _prepare_router(case, g):
    T, E, K, S = case["T"], case["E"], case["K"], case["S"]
    bias = torch.randn(E, generator=g, device="cuda")  # popular and unpopular experts
    logits = (torch.randn(T, E, generator=g, device="cuda") + bias).to(DTYPE[case["dtype"]])
    top = torch.topk(logits.float(), K, dim=1)
    s = {"case": case, "logits": logits, "ids": top.indices.to(torch.int32).contiguous(),
         "w": torch.softmax(top.values, dim=1).contiguous(), "mask": None, "offsets": None}
    # the gradient that the layer's output sends to its routing scores
    s["dw"] = torch.randn(T, K, generator=g, device="cuda") * (1e-2 / T)
    if S > 1:
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
    if case["mask"]:
        s["mask"] = torch.rand(T, generator=g, device="cuda") < 0.85
    if case["op"] == "router_step":
        s["dlogits"] = torch.empty_like(logits)
    return s


def _prepare_distill(case, g):
    N, V, k = case["N"], case["V"], case["k"]
    logits = _vocab_logits(case, g)
    s = {"case": case, "logits": logits, "t_lse": None}
    s["t_ids"] = torch.empty(N, k, dtype=torch.int32, device="cuda")
    s["t_logits"] = torch.empty(N, k, dtype=torch.float32, device="cuda")
    if case["full"]:
        s["t_lse"] = torch.empty(N, device="cuda")
    ban = torch.rand(V, generator=g, device="cuda") < case["banned"] if case["banned"] else None
    if ban is not None:
        ban[:k] = False
    for r in range(0, N, _chunk(V)):
        rows = logits[r:r + _chunk(V)]
        if ban is not None:
            rows.masked_fill_(ban, -math.inf)
        t = rows.float() + 0.5 * torch.randn(rows.shape, generator=g, device="cuda")
        top = torch.topk(t, k, dim=1)
        s["t_ids"][r:r + _chunk(V)] = top.indices.to(torch.int32)
        s["t_logits"][r:r + _chunk(V)] = top.values
        if case["full"]:
            s["t_lse"][r:r + _chunk(V)] = torch.logsumexp(t / case["tau"], dim=1)
    if case["op"] == "distill_grad":
        live = torch.rand(N, generator=g, device="cuda") < 0.95  # prompt tokens carry no loss
        s["weight"] = live.float() * (1024.0 / N)
        s["dlogits"] = torch.empty(N, V, dtype=logits.dtype, device="cuda")
    return s


def _prepare_policy(case, g):
    N, V = case["N"], case["V"]
    logits = _vocab_logits(case, g)
    actions = torch.randint(V, (N,), generator=g, device="cuda")
    boost = 8.0 + 8.0 * torch.rand(N, generator=g, device="cuda")
    row = torch.arange(N, device="cuda")
    logits[row, actions] = boost.to(logits.dtype)  # chosen tokens are likely ones
    s = {"case": case, "logits": logits}
    if case["op"] != "logp":
        lp = torch.empty(N, device="cuda")
        for r in range(0, N, _chunk(V)):
            z = logits[r:r + _chunk(V)].float() / case["tau"]
            a = actions[r:r + _chunk(V)].unsqueeze(1)
            lp[r:r + _chunk(V)] = z.gather(1, a).squeeze(1) - torch.logsumexp(z, 1)
        s["old"] = lp + 0.2 * torch.randn(N, generator=g, device="cuda")
        s["ref"] = lp + 0.4 * torch.randn(N, generator=g, device="cuda") if case["ref"] else None
        s["adv"] = torch.randn(N, generator=g, device="cuda")
    if case["op"] == "policy_grad":
        s["weight"] = torch.full((N,), 1024.0 / N, device="cuda")
        s["dlogits"] = torch.empty(N, V, dtype=logits.dtype, device="cuda")
    # rows of the prompt have no chosen token
    s["actions"] = torch.where(torch.rand(N, generator=g, device="cuda") < 0.06, -1,
                               actions).to(torch.int32)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    group = case["op"].split("_")[0]
    if group == "router":
        return _prepare_router(case, g)
    return _prepare_distill(case, g) if group == "distill" else _prepare_policy(case, g)


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import nvfp4_token_routed_gb300 as M
    c = s["case"]
    op = c["op"]
    if op.startswith("router"):
        losses, counts, tokens = M.router_loss(s["logits"], s["ids"], BALANCE_COEF, Z_COEF,
                                               seq_offsets=s["offsets"], token_mask=s["mask"])
        out = {"losses": losses, "counts": counts, "tokens": tokens}
        if op == "router_step":
            out["dlogits"] = M.router_loss_grad(s["logits"], s["ids"], counts, tokens,
                                                BALANCE_COEF, Z_COEF, seq_offsets=s["offsets"],
                                                token_mask=s["mask"], topk_w=s["w"],
                                                d_topk_w=s["dw"], dlogits=s["dlogits"])
        return out
    if op == "distill_loss":
        return {"loss": M.distill_loss(s["logits"], s["t_ids"], s["t_logits"],
                                       teacher_lse=s["t_lse"], temperature=c["tau"])}
    if op == "distill_grad":
        loss, dlogits = M.distill_loss_grad(s["logits"], s["t_ids"], s["t_logits"], s["weight"],
                                            teacher_lse=s["t_lse"], temperature=c["tau"],
                                            dlogits=s["dlogits"])
        return {"loss": loss, "dlogits": dlogits}
    if op == "logp":
        return {"logp": M.token_logp(s["logits"], s["actions"], temperature=c["tau"])}
    kw = dict(ref_logp=s["ref"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
              kl_coef=KL_COEF if c["ref"] else 0.0, temperature=c["tau"])
    if op == "policy_loss":
        loss, logp = M.policy_loss(s["logits"], s["actions"], s["old"], s["adv"], **kw)
        return {"loss": loss, "logp": logp}
    loss, logp, dlogits = M.policy_loss_grad(s["logits"], s["actions"], s["old"], s["adv"],
                                             s["weight"], dlogits=s["dlogits"], **kw)
    return {"loss": loss, "logp": logp, "dlogits": dlogits}


def _softmax_parts(z):
    """exp(z - max) over the last dimension, its sum and the log of the sum of exp(z)."""
    m = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(dim=1, keepdim=True)
    return e, total, m + torch.log(total)


def _plain_router(s):
    c = s["case"]
    T, E, K, S = c["T"], c["E"], c["K"], c["S"]
    dev = s["logits"].device
    e, total, lse = _softmax_parts(s["logits"].float())
    P, lse = e / total, lse.squeeze(1)
    live = s["mask"].float() if s["mask"] is not None else torch.ones(T, device=dev)
    if s["offsets"] is not None:
        rows = torch.arange(T, device=dev, dtype=torch.int32)
        seg = torch.searchsorted(s["offsets"], rows, right=True) - 1
    else:
        seg = torch.zeros(T, dtype=torch.int64, device=dev)
    n_seg = torch.zeros(S, device=dev).index_add_(0, seg, live)
    n = n_seg.sum()
    P_sum = torch.zeros(S, E, device=dev).index_add_(0, seg, P * live.unsqueeze(1))
    slot = (seg.unsqueeze(1) * E + s["ids"]).reshape(-1)
    one = live.unsqueeze(1).expand(T, K).reshape(-1).to(torch.int32)
    counts = torch.zeros(S * E, dtype=torch.int32, device=dev).index_add_(0, slot, one)
    counts = counts.reshape(S, E)
    f = counts.float() * E / (K * n_seg.clamp_min(1.0)).unsqueeze(1)
    per = 1.0 / n.clamp_min(1.0)
    balance = BALANCE_COEF * per * (f * P_sum).sum()
    z = Z_COEF * per * (live * lse * lse).sum()
    out = {"losses": torch.stack([balance, z]), "counts": counts,
           "tokens": torch.cat([n_seg, n.reshape(1)]).to(torch.int32)}
    if c["op"] == "router_step":
        f_row = f[seg]
        dot = (f_row * P).sum(dim=1, keepdim=True)
        d = P * per * (BALANCE_COEF * (f_row - dot) + 2.0 * Z_COEF * lse.unsqueeze(1))
        w, dw = s["w"], s["dw"]
        d.scatter_add_(1, s["ids"].long(), w * (dw - (w * dw).sum(dim=1, keepdim=True)))
        out["dlogits"] = (d * live.unsqueeze(1)).to(s["logits"].dtype)
    return out


def _plain_distill(s):
    c = s["case"]
    tau = c["tau"]
    e, total, lse = _softmax_parts(s["logits"].float() / tau)
    t = s["t_logits"] / tau
    t_lse = _softmax_parts(t)[2] if s["t_lse"] is None else s["t_lse"].unsqueeze(1)
    q = torch.exp(t - t_lse)
    ids = s["t_ids"].long()
    z_top = s["logits"].gather(1, ids).float() / tau
    loss = tau * tau * (q * ((t - t_lse) - (z_top - lse))).sum(dim=1)
    if c["op"] == "distill_loss":
        return {"loss": loss}
    w = s["weight"].unsqueeze(1)
    loss = torch.where(s["weight"] != 0, loss, 0.0)
    d = e * (w * tau * q.sum(dim=1, keepdim=True) / total)
    d.scatter_add_(1, ids, -w * tau * q)
    return {"loss": loss, "dlogits": d.to(s["logits"].dtype)}


def _plain_policy(s):
    c = s["case"]
    tau = c["tau"]
    live = s["actions"] >= 0
    a = s["actions"].clamp_min(0).long().unsqueeze(1)
    e, total, lse = _softmax_parts(s["logits"].float() / tau)
    logp = (s["logits"].gather(1, a).float() / tau - lse).squeeze(1)
    logp_out = torch.where(live, logp, 0.0)
    if c["op"] == "logp":
        return {"logp": logp_out}
    A = s["adv"]
    ratio = torch.exp(logp - s["old"])
    clipped = ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    loss = -torch.minimum(ratio * A, clipped * A)
    # the clipped branch is constant: it is taken where it is the smaller one
    slope = torch.where(clipped * A < ratio * A, 0.0, -ratio * A)
    if s["ref"] is not None:
        gap = s["ref"] - logp
        loss = loss + KL_COEF * (torch.exp(gap) - gap - 1.0)
        slope = slope + KL_COEF * (1.0 - torch.exp(gap))
    loss = torch.where(live, loss, 0.0)
    if c["op"] == "policy_loss":
        return {"loss": loss, "logp": logp_out}
    slope = (torch.where(live, slope, 0.0) * s["weight"] / tau).unsqueeze(1)
    d = e * (-slope / total)
    d.scatter_add_(1, a, slope)
    return {"loss": loss, "logp": logp_out, "dlogits": d.to(s["logits"].dtype)}


def _run_plain(s):
    group = s["case"]["op"].split("_")[0]
    return {"router": _plain_router, "distill": _plain_distill}.get(group, _plain_policy)(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = torch.empty((), dtype=DTYPE[case["dtype"]]).element_size()
    if case["op"].startswith("router"):
        T, E, K, S = case["T"], case["E"], case["K"], case["S"]
        once = T * E * size + T * K * 4 + (T if case["mask"] else 0)
        n = once + S * (E + 1) * 4 + 12
        flops = T * E * 5.0
        if case["op"] == "router_step":  # a second reading of the logits, as the loss comes before
            n += once + T * K * 8 + T * E * size + S * E * 4
            flops += T * E * 9.0
        return {"bytes": n, "flops": flops}
    N, V = case["N"], case["V"]
    grad = case["op"].endswith("grad")
    n = N * V * size * (2 if grad else 1)
    n += N * (8 * case["k"] + 4 if "k" in case else 24) + (N * 4 if grad else 0)
    return {"bytes": n, "flops": N * V * (6.0 if grad else 4.0)}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    group = case["op"].split("_")[0]
    return {"router": _exact_router, "distill": _exact_distill}.get(group, _exact_policy)(case, s)


def _exact_router(case, s):
    T, E, K, S = case["T"], case["E"], case["K"], case["S"]
    x = s["logits"].to(torch.float64)
    cuts = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    live = torch.ones(T, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"]
    n = int(live.sum())
    balance = z = torch.zeros((), dtype=torch.float64, device=x.device)
    d = torch.zeros_like(x)
    for q in range(S):
        at = torch.nonzero(live[cuts[q]:cuts[q + 1]]).reshape(-1) + cuts[q]
        if not at.numel():
            continue
        logZ = torch.logsumexp(x[at], dim=1)
        p = torch.exp(x[at] - logZ[:, None])
        share = torch.bincount(s["ids"][at].long().reshape(-1), minlength=E).to(torch.float64)
        share = share * E / (K * at.numel())
        balance = balance + BALANCE_COEF * (p @ share).sum() / n
        z = z + Z_COEF * torch.dot(logZ, logZ) / n
        if case["op"] == "router_step":
            g = BALANCE_COEF * (p * share - p * (p @ share)[:, None]) / n
            g += (2 * Z_COEF / n) * logZ[:, None] * p
            w, dw = s["w"][at].double(), s["dw"][at].double()
            jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
            g.scatter_add_(1, s["ids"][at].long(), torch.einsum("tij,tj->ti", jac, dw))
            d[at] = g
    out = {"losses": torch.stack([balance, z]), "counts": None, "tokens": None}
    if case["op"] == "router_step":
        out["dlogits"] = d
    return out


def _exact_distill(case, s):
    N, V, tau = case["N"], case["V"], case["tau"]
    grad = case["op"] == "distill_grad"
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    d = torch.zeros(N, V, dtype=torch.float64, device="cuda") if grad else None
    step = max(1, (1 << 25) // V)
    for r in range(0, N, step):
        logp = torch.log_softmax(s["logits"][r:r + step].double() / tau, dim=1)
        t = s["t_logits"][r:r + step].double() / tau
        logq = t - (torch.logsumexp(t, 1) if s["t_lse"] is None
                    else s["t_lse"][r:r + step].double())[:, None]
        q, ids = logq.exp(), s["t_ids"][r:r + step].long()
        part = tau ** 2 * (q * (logq - logp.gather(1, ids))).sum(1)
        if grad:
            w = s["weight"][r:r + step].double()
            part = part * (w != 0)
            g = logp.exp() * q.sum(1, keepdim=True)
            g.scatter_add_(1, ids, -q)
            d[r:r + step] = g * (tau * w)[:, None]
        loss[r:r + step] = part
    return {"loss": loss, "dlogits": d} if grad else {"loss": loss}


def _exact_policy(case, s):
    N, V, tau = case["N"], case["V"], case["tau"]
    grad = case["op"] == "policy_grad"
    logp = torch.zeros(N, dtype=torch.float64, device="cuda")
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    d = torch.zeros(N, V, dtype=torch.float64, device="cuda") if grad else None
    step = max(1, (1 << 25) // V)
    for r in range(0, N, step):
        act = s["actions"][r:r + step].long()
        at = torch.nonzero(act >= 0).reshape(-1)
        if not at.numel():
            continue
        act = act[at]
        at = at + r
        lsm = torch.log_softmax(s["logits"][at].double() / tau, dim=1)
        lp = lsm.gather(1, act[:, None])[:, 0]
        logp[at] = lp
        if case["op"] == "logp":
            continue
        A, move = s["adv"][at].double(), lp - s["old"][at].double()
        hi, lo = math.log1p(CLIP_HIGH), math.log1p(-CLIP_LOW)
        outer = torch.where(A >= 0, move > hi, move < lo)  # the clipped side of each sign
        edge = torch.where(A >= 0, 1 + CLIP_HIGH, 1 - CLIP_LOW).double()
        loss_r = -A * torch.where(outer, edge, move.exp())
        slope = torch.where(outer, 0.0, -A * move.exp())
        if s["ref"] is not None:
            gap = s["ref"][at].double() - lp
            loss_r = loss_r + KL_COEF * (torch.expm1(gap) - gap)
            slope = slope - KL_COEF * torch.expm1(gap)
        loss[at] = loss_r
        if grad:
            g = -lsm.exp()
            g[torch.arange(at.numel(), device="cuda"), act] += 1
            d[at] = g * (slope * s["weight"][at].double() / tau)[:, None]
    if case["op"] == "logp":
        return {"logp": logp}
    out = {"loss": loss, "logp": logp}
    if grad:
        out["dlogits"] = d
    return out
