"""W4A4 layers whose stages are reused many times (28 blocks of 256 in a ring of 5 to 8), with
block scales over many magnitudes: the same bits in every run, and the oracle's result."""
import pytest
import torch

import nvfp4_token_routed_gb300 as M
from nvfp4_token_routed_gb300 import workloads as W

from helpers import OracleRun, bf16_np, rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,I,E,K,act", [(6, 256, 8, 4, "swiglu"), (150, 512, 4, 2, "relu2"),
                                         (260, 256, 2, 1, "swiglu")])
def test_scales_of_reused_stages(T, I, E, K, act):
    wl = W.Workload(f"{act}_T{T}_H7168_I{I}_E{E}_K{K}", T, 7168, I, E, K, act)
    g = torch.Generator().manual_seed(T)
    # one magnitude a block of 16 columns, undone by the weights
    mag = torch.exp2(torch.randint(-6, 7, (wl.H // 16,), generator=g).float()).repeat_interleave(16)
    x = (W.make_x(wl).float() * mag).bfloat16()
    w1, w2 = W.make_weights(wl)
    w1 = (w1.float() / mag).bfloat16()
    ids, wts = W.make_routing(wl)
    w = M.prepare_weights(w1.to(DEV), w2.to(DEV), wl.act)
    q = M.quantize_tokens(x.to(DEV))
    ws = M.workspace(w, wl.T, wl.K)
    outs = [M.forward(w, *q, ids.to(DEV), wts.to(DEV), ws=ws).clone() for _ in range(20)]
    assert M.moe_nvfp4_read_status(ws) == 0
    assert all(torch.equal(o, outs[0]) for o in outs)
    want = OracleRun(wl, x, w1, w2, ids, wts).res["out"]
    got = outs[0].cpu().view(torch.int16).numpy().view("uint16")
    assert rel_l2(bf16_np(got), bf16_np(want)) <= 1e-2
