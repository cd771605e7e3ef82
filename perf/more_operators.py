"""Cases for the operators of a differentiable pass through routed 4-bit experts,
their plain forms and their definitions in 64 bits.

Three groups:
  dispatch / combine   routes sorted by expert, token rows copied to their routes'
                       rows and summed back with the routing weights, and the
                       gradients of both
  act / checkpoint     the experts' activation, whose input is kept in 8 bits for
                       the backward pass (E4M3, a power of two per 32 values), the
                       gradient from it, and a row checkpoint written and read back
  product              microscaled FP4 (E2M1, a power of two per 32 values): rows
                       quantised and multiplied with the weights of their expert

`run` takes the framework's kernels where `own` is true, else elementary torch
operations in fp32, rounded once at the end.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3_MAX_EXP, E4M3_FRAC = 8, 0.875  # 448 = 2 * 0.875 * 2^8
E2M1_MAX_EXP, E2M1_FRAC = 2, 0.75   # 6 = 2 * 0.75 * 2^2
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _routes(name, op, T, E, K, H, dtype="bf16", empty=0.0):
    c = {"op": op, "T": T, "E": E, "K": K, "H": H, "dtype": dtype, "empty": empty}
    return dict(c, name=name) if name else c


def _act(name, act, R, I, limit=0.0, dtype="bf16"):
    c = {"op": "act_step", "act": act, "R": R, "I": I, "limit": limit, "dtype": dtype}
    return dict(c, name=name) if name else c


def _checkpoint(name, R, D, dtype="bf16"):
    c = {"op": "checkpoint", "R": R, "D": D, "dtype": dtype}
    return dict(c, name=name) if name else c


def _product(name, R, E, N, D, dtype="bf16"):
    c = {"op": "product", "R": R, "E": E, "N": N, "D": D, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 16 sequences: routes sorted, token rows copied
        _routes("dispatch_T16_E256_H7168", "dispatch", 16, 256, 8, 7168),
        # a training batch of the 384-expert layer: to the experts, and the rows'
        # gradients back to the tokens
        _routes("dispatch_step_T4096_E384_H7168", "dispatch_step", 4096, 384, 6, 7168),
        # the experts' rows back to the tokens, and the gradients of rows and weights
        _routes("combine_step_T4096_E384_H7168", "combine_step", 4096, 384, 6, 7168),
        # a ragged batch whose padding tokens and dropped routes are empty slots, odd rows
        _routes("combine_step_T1531_E60_H1001_f16", "combine_step", 1531, 60, 4, 1001,
                dtype="f16", empty=0.2),
        # a small fine-tuning batch through the experts' activation and back
        _act("act_step_R128_I1024", "swiglu", 128, 1024),
        # a training batch of clamped SwiGLU experts
        _act("act_step_R24576_I2048_clamped", "swiglu", 24576, 2048, limit=10.0),
        # squared ReLU experts of an odd width
        _act("act_step_R5001_I1407_relu2_f16", "relu2", 5001, 1407, dtype="f16"),
        # the residual stream of a layer kept in 8 bits, and read back
        _checkpoint("checkpoint_R4096_D7168", 4096, 7168),
        # FC1 of a decode step: 16 tokens, 8 experts each, of 64
        _product("product_R128_E64_N2048_D2048", 128, 64, 2048, 2048),
        # a shared expert over a prompt: one matrix
        _product("product_R4096_N4096_D7168", 4096, 1, 4096, 7168),
        # FC1 of a training batch over ragged groups
        _product("product_R16384_E32_N4096_D7168", 16384, 32, 4096, 7168),
        # odd groups, outputs and reductions
        _product("product_R517_E5_N1003_D801_f16", 517, 5, 1003, 801, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    group = rng.choice(["routes", "routes", "act", "product", "product", "checkpoint"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if group == "routes":
        E = rng.choice([1, 8, 33, 60, 64, 128, 160, 256, 384, 1000])
        K = rng.choice([k for k in (1, 2, 3, 4, 6, 8, 8) if k <= E])
        H = _log_int(rng, 16, 7168)
        if rng.random() < 0.5:
            H = max(64, H // 64 * 64)
        most = 4096 * 6 * 7168 // (2 if dtype == "f32" else 1)
        T = _log_int(rng, 1, min(32768, most // (K * H)))
        return _routes(None, rng.choice(["dispatch", "dispatch_step", "combine_step"]), T, E, K, H,
                       dtype, rng.choice([0.0, 0.0, 0.15]))
    if group == "act":
        act = rng.choice(["swiglu", "swiglu", "relu2"])
        I = _log_int(rng, 32, 4096)
        if rng.random() < 0.6:
            I = max(64, I // 64 * 64)
        R = _log_int(rng, 1, min(32768, 24576 * 2048 // I // (2 if dtype == "f32" else 1)))
        limit = rng.choice([0.0, 7.0]) if act == "swiglu" else 0.0
        return _act(None, act, R, I, limit, dtype)
    if group == "checkpoint":
        D = _log_int(rng, 32, 7168)
        return _checkpoint(None, _log_int(rng, 1, min(32768, 4096 * 7168 // D)), D, dtype)
    D = _log_int(rng, 32, 7168)
    N = _log_int(rng, 16, 4096)
    if rng.random() < 0.6:
        D, N = max(64, D // 64 * 64), max(64, N // 64 * 64)
    E = rng.choice([1, 1, 3, 8, 16, 32])
    return _product(None, _log_int(rng, 1, 16384), E, N, D, rng.choice(["bf16", "bf16", "f16"]))


# ------------------------------------------------------------------ inputs

def _ids(case, g):
    """Top-K of router logits with popular and unpopular experts; -1 in empty slots."""
    T, E, K = case["T"], case["E"], case["K"]
    z = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g,
                                                                          device="cuda")
    top = torch.topk(z, K, dim=1)
    ids, w = top.indices.to(torch.int32), torch.softmax(top.values, dim=1)
    if case["empty"]:
        ids = torch.where(torch.rand(T, K, generator=g, device="cuda") < case["empty"], -1, ids)
    return ids.contiguous(), w.contiguous()


def _randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(DTYPE[dtype])


def _prepare_routes(case, g):
    T, K, H, dt = case["T"], case["K"], case["H"], case["dtype"]
    ids, w = _ids(case, g)
    s = {"case": case, "ids": ids}
    # rows behind the last route stay as they were: the buffers of a program's first step
    if case["op"] == "combine_step":
        s.update(w=w, rows=_randn(g, T * K, H, dtype=dt), dout=_randn(g, T, H, dtype=dt),
                 drows=torch.zeros(T * K, H, dtype=DTYPE[dt], device="cuda"))
        s["plan"] = _plain_sort(ids, case["E"])
        return s
    s.update(x=_randn(g, T, H, dtype=dt),
             rows=torch.zeros(T * K, H, dtype=DTYPE[dt], device="cuda"))
    if case["op"] == "dispatch_step":
        s["drows"] = _randn(g, T * K, H, dtype=dt)
    return s


def _prepare_act(case, g):
    R, I, dt = case["R"], case["I"], case["dtype"]
    width = 2 * I if case["act"] == "swiglu" else I
    spread = torch.exp(0.5 * torch.randn(R, 1, generator=g, device="cuda"))
    h = torch.randn(R, width, generator=g, device="cuda") * (2.0 * spread)
    h = h.to(DTYPE[dt])
    return {"case": case, "h": h, "dy": _randn(g, R, I, dtype=dt, scale=0.1)}


def _prepare_checkpoint(case, g):
    x = torch.randn(case["R"], case["D"], generator=g, device="cuda")
    loud = torch.rand(case["D"], generator=g, device="cuda") < 0.01  # channels that stand out
    return {"case": case, "x": torch.where(loud, x * 20.0, x).to(DTYPE[case["dtype"]])}


def _prepare_product(case, g):
    R, E, N, D = case["R"], case["E"], case["N"], case["D"]
    Dp = (D + 255) // 256 * 256
    codes = torch.zeros(E * N, Dp // 2, dtype=torch.uint8, device="cuda")
    rows_p = (E * N + 1) // 2 * 2
    scales = torch.zeros(Dp // 256, rows_p, 8, dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.zeros(N, Dp, device="cuda")
        w[:, :D] = torch.randn(N, D, generator=g, device="cuda") * D ** -0.5
        mag, exp = _plain_e2m1(w.reshape(N, Dp // 32, 32))
        code = torch.searchsorted(torch.tensor(E2M1, device="cuda"), mag.abs().contiguous())
        code = (code + 8 * torch.signbit(mag)).to(torch.uint8).reshape(N, Dp // 2, 2)
        codes[e * N:(e + 1) * N] = code[..., 0] | (code[..., 1] << 4)
        at = (exp + 127).to(torch.uint8).reshape(N, Dp // 256, 8).transpose(0, 1)
        scales[:, e * N:(e + 1) * N] = at
    s = {"case": case, "codes": codes, "scales": scales,
         "x": _randn(g, R, D, dtype=case["dtype"]), "offsets": None}
    if E > 1:
        p = torch.softmax(0.5 * torch.randn(E, generator=g, device="cuda"), 0)
        load = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=E)
        s["offsets"] = torch.cat([load.new_zeros(1), load.cumsum(0)]).to(torch.int32)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"act_step": _prepare_act, "checkpoint": _prepare_checkpoint,
            "product": _prepare_product}.get(case["op"], _prepare_routes)(case, g)


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import nvfp4_token_routed_gb300 as M
    c = s["case"]
    op = c["op"]
    if op.startswith("dispatch"):
        plan = M.sort_routes(s["ids"], c["E"])
        out = {"offsets": plan.offsets, "perm": plan.perm, "inv": plan.inv,
               "rows": M.dispatch(s["x"], plan, rows=s["rows"])}
        if op == "dispatch_step":
            out["dx"] = M.dispatch_grad(s["drows"], plan)
        return out
    if op == "combine_step":
        plan = M.RoutePlan(*s["plan"])
        out = M.combine(s["rows"], plan, s["w"])
        drows, dw = M.combine_grad(s["rows"], plan, s["w"], s["dout"], drows=s["drows"])
        return {"out": out, "drows": drows, "dw": dw}
    if op == "act_step":
        y, kept = M.expert_act(s["h"], c["act"], swiglu_limit=c["limit"], checkpoint=True)
        return {"y": y, "dh": M.expert_act_grad(kept, s["dy"])}
    if op == "checkpoint":
        return {"x": M.restore(M.checkpoint(s["x"]))}
    w = M.MxTensor(s["codes"], s["scales"], (c["E"], c["N"], c["D"]))
    return {"y": M.mx_product(M.mx_quantize(s["x"]), w, offsets=s["offsets"],
                              dtype=s["x"].dtype)}


def _plain_sort(ids, E):
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True).to(torch.int32)
    count = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    count.index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([count.new_zeros(1), count[:E].cumsum(0)]).to(torch.int32)
    at = torch.arange(flat.numel(), dtype=torch.int32, device=ids.device)
    inv = torch.empty_like(at)
    inv[order.long()] = torch.where(at < offsets[E], at, -1)
    return offsets, torch.where(at < offsets[E], order, -1), inv.reshape(ids.shape)


def _route_rows(rows, inv, k):
    """Row of each token's k-th route in fp32, zeros where the slot is empty."""
    at = inv[:, k]
    return torch.where((at >= 0).unsqueeze(1), rows[at.clamp_min(0).long()].float(), 0.0)


def _plain_routes(s):
    c = s["case"]
    K = c["K"]
    if c["op"] == "combine_step":
        _, perm, inv = s["plan"]
        live = perm >= 0
        at = perm.clamp_min(0).long()
        out = torch.zeros(c["T"], c["H"], device=perm.device)
        dw = torch.empty(c["T"], K, device=perm.device)
        dout = s["dout"].float()
        for k in range(K):
            y = _route_rows(s["rows"], inv, k)
            out += s["w"][:, k:k + 1] * y
            dw[:, k] = (y * dout).sum(1)
        wr = s["w"].reshape(-1)[at].unsqueeze(1)
        drows = (wr * dout[at // K]).to(s["rows"].dtype)
        s["drows"].copy_(torch.where(live.unsqueeze(1), drows, s["drows"]))
        return {"out": out.to(s["rows"].dtype), "drows": s["drows"], "dw": dw}
    offsets, perm, inv = _plain_sort(s["ids"], c["E"])
    at = perm.clamp_min(0).long() // K
    s["rows"].copy_(torch.where((perm >= 0).unsqueeze(1), s["x"][at], s["rows"]))
    res = {"offsets": offsets, "perm": perm, "inv": inv, "rows": s["rows"]}
    if c["op"] == "dispatch_step":
        dx = torch.zeros(c["T"], c["H"], device=perm.device)
        for k in range(K):
            dx += _route_rows(s["drows"], inv, k)
        res["dx"] = dx.to(s["drows"].dtype)
    return res


def _plain_blocks(x, max_exp, frac):
    """Exponent of each block of 32 along the last dimension: the smallest with which no
    value passes the element type's largest."""
    m, k = torch.frexp(x.abs().amax(dim=-1, keepdim=True))
    return torch.clamp(k - 1 - max_exp + (m > frac).to(k.dtype), -127, 127)


def _plain_e2m1(x):
    """Values of the elements (before their scale) and the blocks' exponents."""
    exp = _plain_blocks(x, E2M1_MAX_EXP, E2M1_FRAC)
    v = torch.ldexp(x, -exp)
    mag = v.abs()
    step = torch.where(mag >= 4.0, 2.0, torch.where(mag >= 2.0, 1.0, 0.5))
    return torch.copysign(torch.round(mag / step) * step, v), exp


def _plain_e4m3(x):
    """[R, D] rounded to what 8 bits hold, in fp32."""
    R, D = x.shape
    pad = torch.zeros(R, (D + 31) // 32 * 32, device=x.device)
    pad[:, :D] = x
    blocks = pad.reshape(R, -1, 32)
    exp = _plain_blocks(blocks, E4M3_MAX_EXP, E4M3_FRAC)
    q = torch.ldexp(blocks, -exp).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, exp).reshape(R, -1)[:, :D]


def _plain_act(s):
    c = s["case"]
    I, L, dt = c["I"], c["limit"], s["h"].dtype
    h, dy = s["h"].float(), s["dy"].float()
    if c["act"] == "relu2":
        return {"y": h.clamp_min(0.0).square().to(dt),
                "dh": (2.0 * dy * _plain_e4m3(h).clamp_min(0.0)).to(dt)}
    g, u = h[:, :I], h[:, I:]
    if L:
        g, u = g.clamp_max(L), u.clamp(-L, L)
    y = g / (1.0 + torch.exp(-g)) * u
    g, u = _plain_e4m3(h[:, :I]), _plain_e4m3(h[:, I:])
    g_in = u_in = 1.0
    if L:
        g_in, u_in = (g <= L).float(), (u.abs() <= L).float()
        g, u = g.clamp_max(L), u.clamp(-L, L)
    sig = 1.0 / (1.0 + torch.exp(-g))
    dg = dy * u * sig * (1.0 + g * (1.0 - sig)) * g_in
    du = dy * g * sig * u_in
    return {"y": y.to(dt), "dh": torch.cat([dg, du], dim=1).to(dt)}


def _unpack(case, codes, scales, e):
    """Weights of expert e in fp32 [N, D] from codes and scales."""
    N, D = case["N"], case["D"]
    c = codes[e * N:(e + 1) * N]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=c.device)
    v = table[torch.stack([c & 15, c >> 4], dim=2).reshape(N, -1).int()]
    exp = scales[:, e * N:(e + 1) * N].transpose(0, 1).reshape(N, -1, 1).int() - 127
    return torch.ldexp(v.reshape(N, -1, 32), exp).reshape(N, -1)[:, :D]


def _plain_product(s):
    c = s["case"]
    R, E, N, D = c["R"], c["E"], c["N"], c["D"]
    x = torch.zeros(R, (D + 31) // 32 * 32, device="cuda")
    x[:, :D] = s["x"]
    v, exp = _plain_e2m1(x.reshape(R, -1, 32))
    q = torch.ldexp(v, exp).reshape(R, -1)[:, :D]
    cuts = [0, R] if s["offsets"] is None else s["offsets"].tolist()
    y = torch.empty(R, N, device="cuda")
    for e in range(E):
        if cuts[e] < cuts[e + 1]:
            y[cuts[e]:cuts[e + 1]] = q[cuts[e]:cuts[e + 1]] @ _unpack(c, s["codes"], s["scales"],
                                                                      e).t()
    return {"y": y.to(s["x"].dtype)}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "checkpoint":
        return {"x": _plain_e4m3(s["x"].float()).to(s["x"].dtype)}
    return {"act_step": _plain_act, "product": _plain_product}.get(op, _plain_routes)(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = torch.empty((), dtype=DTYPE[case["dtype"]]).element_size()
    op = case["op"]
    if op in ("dispatch", "dispatch_step", "combine_step"):
        T, K, H, E = case["T"], case["K"], case["H"], case["E"]
        live = T * K * (1.0 - case["empty"])
        rows, tokens = live * H * size, T * H * size
        if op == "combine_step":  # forward, and rows a second time for the weights' gradient
            n = rows + tokens + T * K * 8 + rows + tokens + rows + T * K * 12
            return {"bytes": n, "flops": live * H * 5.0}
        n = tokens + rows + T * K * 12 + E * 4
        if op == "dispatch_step":
            return {"bytes": n + rows + tokens + T * K * 4, "flops": live * H * 1.0}
        return {"bytes": n, "flops": 0.0}
    if op == "act_step":
        R, I = case["R"], case["I"]
        W = 2 * I if case["act"] == "swiglu" else I
        kept = R * W * (1.0 + 1.0 / 32)  # written, then read
        return {"bytes": 2 * R * (W + I) * size + 2 * kept, "flops": R * W * 14.0}
    R, D = case["R"], case["D"]
    if op == "checkpoint":
        return {"bytes": 2 * R * D * size + 2 * R * D * (1.0 + 1.0 / 32), "flops": R * D * 4.0}
    N, used = case["N"], min(case["E"], R)
    n = used * N * D * 17 / 32 + R * D * size + R * N * size
    return {"bytes": n, "flops": 2.0 * R * N * D}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        return {"x": _exact_held(s["x"], 448.0, 3, -6)}
    return {"act_step": _exact_act, "product": _exact_product}.get(op, _exact_routes)(case, s)


def _exact_held(x, largest, frac_bits, least_exp):
    """x [R, D] at what a format with blocks of 32 holds of it: elements of `frac_bits`
    fraction bits, exponents from `least_exp`, times the smallest power of two that keeps
    the block's largest value within `largest`."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    D = x.shape[1]
    for j in range(0, D, 32 * 64):
        w = x[:, j:j + 32 * 64].double()
        full = torch.nn.functional.pad(w, (0, -w.shape[1] % 32)).unflatten(1, (-1, 32))
        top = full.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2(top / largest)).nan_to_num(neginf=-127.0)
        e = e + (top > largest * torch.exp2(e)).double()          # the logarithm's rounding
        e = e - (top <= largest * torch.exp2(e - 1)).double()
        unit = torch.exp2(e.clamp(-127.0, 127.0))
        v = full / unit
        ulp = torch.frexp(v)[1].double() - 1                        # floor(log2 |v|)
        ulp = torch.exp2(torch.where(v == 0, float(least_exp), ulp).clamp_min(least_exp)
                         - frac_bits)
        out[:, j:j + 32 * 64] = (torch.round(v / ulp) * ulp * unit).flatten(1)[:, :w.shape[1]]
    return out


def _exact_act(case, s):
    I, L = case["I"], case["limit"]
    dy = s["dy"].double()
    if case["act"] == "relu2":
        h = s["h"].double()
        kept = _exact_held(s["h"], 448.0, 3, -6)
        return {"y": torch.where(h > 0, h * h, 0.0), "dh": torch.where(kept > 0, 2 * kept, 0.0) * dy}
    bound = L if L else math.inf
    g, u = s["h"][:, :I].double().clamp(max=bound), s["h"][:, I:].double().clamp(-bound, bound)
    y = g * torch.sigmoid(g) * u
    g = _exact_held(s["h"][:, :I], 448.0, 3, -6)
    u = _exact_held(s["h"][:, I:], 448.0, 3, -6)
    gc, uc = g.clamp(max=bound), u.clamp(-bound, bound)
    p = torch.sigmoid(gc)
    dg = torch.where(g > bound, 0.0, dy * uc * (p + gc * p * torch.sigmoid(-gc)))
    du = torch.where(u.abs() > bound, 0.0, dy * gc * p)
    return {"y": y, "dh": torch.cat([dg, du], 1)}


def _exact_product(case, s):
    R, E, N, D = case["R"], case["E"], case["N"], case["D"]
    q = _exact_held(s["x"], 6.0, 1, 0)
    bounds = torch.tensor([0, R]) if s["offsets"] is None else s["offsets"].cpu()
    y = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    value = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = int(bounds[e]), int(bounds[e + 1])
        if a == b:
            continue
        packed = s["codes"][e * N:(e + 1) * N].long()
        w = torch.zeros(N, packed.shape[1] * 2, dtype=torch.float64, device="cuda")
        for half, nibble in ((0, packed % 16), (1, packed // 16)):
            w[:, half::2] = value[nibble % 8] * (1.0 - 2.0 * (nibble // 8).double())
        unit = torch.exp2(s["scales"][:, e * N:(e + 1) * N].permute(1, 0, 2).flatten(1).double()
                          - 127.0)
        w *= unit.repeat_interleave(32, dim=1)
        y[a:b] = q[a:b] @ w[:, :D].t()
    return {"y": y}


def _exact_routes(case, s):
    T, E, K, H = case["T"], case["E"], case["K"], case["H"]
    ids = s["ids"].reshape(-1).tolist()
    groups = [[] for _ in range(E)]
    for i, e in enumerate(ids):
        if 0 <= e < E:
            groups[e].append(i)
    perm = torch.tensor([i for grp in groups for i in grp], dtype=torch.int64, device="cuda")
    token = perm // K
    n = perm.numel()
    if case["op"] == "combine_step":
        w = s["w"].reshape(-1).double()[perm]
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T * K, dtype=torch.float64, device="cuda")
        drows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
        for r in range(0, n, 4096):
            y, at = s["rows"][r:r + 4096][:n - r].double(), token[r:r + 4096]
            d = s["dout"][at].double()
            out.index_add_(0, at, w[r:r + 4096, None] * y)
            dw[perm[r:r + 4096]] = torch.einsum("rh,rh->r", y, d)
            drows[r:r + y.shape[0]] = w[r:r + 4096, None] * d
        return {"out": out, "drows": drows, "dw": dw.reshape(T, K)}
    rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    rows[:n] = s["x"][token].double()
    res = {"offsets": None, "perm": None, "inv": None, "rows": rows}
    if case["op"] == "dispatch_step":
        dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for r in range(0, n, 4096):
            dx.index_add_(0, token[r:r + 4096], s["drows"][r:r + 4096][:n - r].double())
        res["dx"] = dx
    return res
