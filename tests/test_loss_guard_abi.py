"""Argument checks of the losses' failure self-test, without a GPU."""
import pytest

import nvfp4_token_routed_gb300 as M

P = 4096  # a non-null, aligned pointer that nothing looks at


@pytest.fixture(scope="module")
def lib():
    from nvfp4_token_routed_gb300 import build
    build.build()
    return M.lib()


@pytest.mark.parametrize("kw,code", [
    (dict(role=-1), 1), (dict(role=4), 1), (dict(rank=-1), 1), (dict(row=-1), 1),
    (dict(cols=8192), 2), (dict(dtype=0), 2), (dict(rank=2), 1), (dict(cols=30000, rank=1), 1),
    (dict(out=None), 1), (dict(out=P + 1), 3), (dict(rows=0, out=None), 0)])
def test_refusals(lib, kw, code):
    a = dict(role=0, rank=0, row=0, cols=80000, dtype=1, out=P, rows=4)
    a.update(kw)
    z = M.moe_logits(P, a["cols"], a["rows"], a["cols"], a["dtype"])
    assert lib.moe_nvfp4_selftest_loss_timeout(z, P, 0, P, P, a["role"], a["rank"], a["row"], P, P,
                                               a["out"], a["cols"], None) == code
