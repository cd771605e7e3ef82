"""Plain definitions in 64 bits of the routed-row operators, on the CPU.

Nothing here uses the library: sorting, rows, blocks of 32 with a power of two, the
activations and their gradients, and products, each from its formula.
"""
import math

import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3_MAX, E2M1_MAX = 448.0, 6.0


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the type's smallest step: what rounding costs values below its normal range."""
    info = torch.finfo(dtype)
    return info.smallest_normal * info.eps / 2


def sort(ids, E):
    flat = [int(e) for e in ids.reshape(-1)]
    order = [i for e in range(E) for i, x in enumerate(flat) if x == e]
    offsets = [0]
    for e in range(E):
        offsets.append(offsets[-1] + sum(x == e for x in flat))
    inv = torch.full((len(flat),), -1, dtype=torch.int32)
    for r, i in enumerate(order):
        inv[i] = r
    perm = torch.full((len(flat),), -1, dtype=torch.int32)
    perm[:len(order)] = torch.tensor(order, dtype=torch.int32)
    return torch.tensor(offsets, dtype=torch.int32), perm, inv.reshape(ids.shape)


def combine(rows, inv, w):
    """out and the sum of the terms' magnitudes."""
    T, K = inv.shape
    out = torch.zeros(T, rows.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for t in range(T):
        for k in range(K):
            r = int(inv[t, k])
            if r >= 0:
                term = (1.0 if w is None else float(w[t, k])) * rows[r].double()
                out[t] += term
                mag[t] += term.abs()
    return out, mag


def combine_grad(rows, inv, w, dout):
    """drows (zeros where no route lies), dw and the sum of dw's terms' magnitudes."""
    T, K = inv.shape
    drows = torch.zeros(rows.shape, dtype=torch.float64)
    dw, mag = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            r = int(inv[t, k])
            if r >= 0:
                d = dout[t].double()
                drows[r] = (1.0 if w is None else float(w[t, k])) * d
                dw[t, k] = (rows[r].double() * d).sum()
                mag[t, k] = (rows[r].double() * d).abs().sum()
    return drows, dw, mag


def blocks(x, largest):
    """x [R, D] padded to whole blocks [R, B, 32] in 64 bits, and each block's exponent: the
    smallest e in [-127, 127] with max |x| <= largest * 2^e; None for a block with an
    infinity or a NaN."""
    pad = torch.nn.functional.pad(x.double(), (0, -x.shape[1] % 32)).unflatten(1, (-1, 32))
    exps = []
    for row in pad:
        exps.append([])
        for b in row:
            if not bool(torch.isfinite(b).all()):
                exps[-1].append(None)
                continue
            top, e = float(b.abs().max()), -127
            if top > 0:
                e = math.frexp(top / largest)[1] - 2
                while top > largest * 2.0 ** e:
                    e += 1
                e = max(e, -127)
            exps[-1].append(e)
    return pad, exps


def held(x, largest, fraction_bits, least_exp, most=math.inf):
    """(values that the format holds of x [R, D], scale bytes [R, B]); a value that would round
    past `most` rounds down."""
    pad, exps = blocks(x, largest)
    unit = torch.tensor([[math.nan if e is None else 2.0 ** e for e in row] for row in exps],
                        dtype=torch.float64).unsqueeze(2)
    byte = torch.tensor([[255 if e is None else e + 127 for e in row] for row in exps])
    v = pad / unit
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** (least_exp - 1))))
    e = torch.where(2.0 ** (e + 1) <= v.abs(), e + 1, torch.where(2.0 ** e > v.abs(), e - 1, e))
    step = 2.0 ** (e.clamp_min(least_exp) - fraction_bits)
    q = torch.round(v / step) * step
    q = torch.where((q * unit).abs() > most, torch.sign(v) * (torch.floor(v.abs() / step) * step), q)
    return (q * unit).flatten(1)[:, :x.shape[1]], byte.to(torch.uint8)


def held8(x):
    return held(x, E4M3_MAX, 3, -6, torch.finfo(x.dtype).max)


def held4(x):
    return held(x, E2M1_MAX, 1, 0)


def act(h, act, limit):
    h = h.double()
    if act == "relu2":
        return h.clamp_min(0.0) ** 2
    I = h.shape[1] // 2
    L = limit if limit else math.inf
    g, u = h[:, :I].clamp(max=L), h[:, I:].clamp(-L, L)
    return g * torch.sigmoid(g) * u


def kept(h, act):
    if act == "relu2":
        return held8(h)[0]
    I = h.shape[1] // 2
    return torch.cat([held8(h[:, :I])[0], held8(h[:, I:])[0]], 1)


def act_grad(h, act, limit, dy):
    """Gradient at h (64 bits), and the bound's weight of each element."""
    dy = dy.double()
    if act == "relu2":
        d = 2.0 * dy * h.clamp_min(0.0)
        return d, d.abs()
    I = h.shape[1] // 2
    L = limit if limit else math.inf
    g0, u0 = h[:, :I], h[:, I:]
    g, u = g0.clamp(max=L), u0.clamp(-L, L)
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    dg = torch.where(g0 > L, 0.0, dy * u * s * (1.0 + g * r))
    du = torch.where(u0.abs() > L, 0.0, dy * g * s)
    # s is off by (5 + 1.2 |g|) 2^-23 of itself, which multiplies 1 + g (1 - s); 1 - s by 3 2^-23,
    # which g multiplies; below 2^-126 (g < -87) s may be 0: 2^-125 is 2^-102 of 2^-23
    wide = 12.0 + 4.0 * g.abs()
    return torch.cat([dg, du], 1), torch.cat(
        [(wide * (1.0 + g.abs() * r) * s + 2.0 ** -102 * (1.0 + g.abs())) * (dy * u).abs(),
         wide * du.abs() + 2.0 ** -102 * (dy * g).abs()], 1)
