"""Products whose stages are reused many times, every stage with scales of its own: a scale
that is staged before the MMAs of the stage's last use have read theirs would show.

The values make the result exact: x = +-2^i or 0, w = +-2^j or 0 with 0 <= i, j <= 3 and one
exponent a block of 32, so both are held exactly, every term is an integer of at most 2^6, and
a sum of 65536 of them stays below 2^24.
"""
import pytest
import torch

import nvfp4_token_routed_gb300 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _powers(rows, D, g):
    sign = torch.randint(-1, 2, (rows, D), generator=g, device=DEV).float()
    exps = torch.randint(0, 4, (rows, (D + 31) // 32), generator=g, device=DEV)
    return sign * torch.exp2(exps.float()).repeat_interleave(32, 1)[:, :D]


# rows a group, experts, outputs, length: single blocks with two, four and many stages in
# flight, then pairs with one accumulator and with two
@pytest.mark.parametrize("rows,E,N,D", [(3, 1, 300, 65536), (64, 2, 130, 30000),
                                        (190, 3, 257, 16384), (7, 40, 640, 4096),
                                        (256, 4, 2560, 8192), (1000, 2, 2700, 16000),
                                        (229, 5, 2436, 4096)])
def test_scales_of_reused_stages(rows, E, N, D):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + D)
    x, w = _powers(rows * E, D, g), _powers(E * N, D, g)
    q, qw = M.mx_quantize(x), M.mx_quantize(w.view(E, N, D))
    offsets = torch.arange(0, rows * E + 1, rows, dtype=torch.int32, device=DEV)
    want = torch.cat([x[e * rows:(e + 1) * rows].double() @ w[e * N:(e + 1) * N].double().t()
                      for e in range(E)])
    for _ in range(5):
        got = M.mx_product(q, qw, offsets, torch.float32)
        assert torch.equal(got.double(), want)


def test_products_one_behind_the_other():
    """Launches of pairs and of single blocks in turn, hundreds without a pause: what one leaves
    in flight at its end would meet the next one's barriers."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    E, N, D = 4, 2560, 2048
    qw = M.mx_quantize(_powers(E * N, D, g).view(E, N, D))
    many, few = M.mx_quantize(_powers(1024, D, g)), M.mx_quantize(_powers(20, D, g))
    cut = [torch.tensor(o, dtype=torch.int32, device=DEV) for o in ([0, 256, 512, 768, 1024],
                                                                   [0, 9, 9, 19, 20])]
    want = [M.mx_product(many, qw, cut[0]), M.mx_product(few, qw, cut[1])]
    outs = [torch.empty_like(w) for w in want]
    for _ in range(300):
        for o in outs:
            o.fill_(7.0)
        M.mx_product(many, qw, cut[0], out=outs[0])
        M.mx_product(few, qw, cut[1], out=outs[1])
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
