"""The training objectives' entry points without a GPU: argument checks answer before
any CUDA call, and calls without rows succeed."""
import pytest

import nvfp4_token_routed_gb300 as M

P = 4096  # a non-null, aligned pointer that nothing looks at


@pytest.fixture(scope="module")
def lib():
    from nvfp4_token_routed_gb300 import build
    build.build()
    return M.lib()


def _z(rows=4, cols=100, ld=None, data=P, dtype=0):
    return M.moe_logits(data, cols if ld is None else ld, rows, cols, dtype)


def _t(ids=P, logits=P, lse=None, K=3, i64=0, dtype=0):
    return M.moe_teacher(ids, logits, lse, K, i64, dtype)


def test_logits_checks(lib):
    def logp(z, actions=P, i64=0, tau=1.0, out=P):
        return lib.moe_nvfp4_token_logp(z, actions, i64, tau, out, None)

    assert logp(_z(rows=0, data=None), None, out=None) == 0
    assert lib.moe_nvfp4_token_logp(None, P, 0, 1.0, P, None) == 1
    for z, code in ((_z(rows=-1), 1), (_z(cols=0), 1), (_z(dtype=3), 1), (_z(dtype=-1), 1),
                    (_z(ld=99), 1), (_z(data=None), 1), (_z(cols=(1 << 18) + 1), 2),
                    (_z(rows=(1 << 26) + 1), 2), (_z(data=P + 2), 3), (_z(data=P + 1, dtype=1), 3)):
        assert logp(z) == code
    assert logp(_z(), actions=None) == 1 and logp(_z(), out=None) == 1
    assert logp(_z(), actions=P + 2) == 3 and logp(_z(), actions=P + 4, i64=1) == 3
    assert logp(_z(), out=P + 2) == 3 and logp(_z(), i64=2) == 1
    for tau in (0.0, -1.0, float("inf"), float("nan"), 1e-38):
        assert logp(_z(), tau=tau) == 1


def test_policy_checks(lib):
    def call(lo=0.2, hi=0.2, kl=0.0, tau=1.0, ref=None, w=None, d=P, ld=100, z=None, old=P):
        o = M.moe_policy_opts(lo, hi, kl, tau)
        return lib.moe_nvfp4_policy_loss_grad(z or _z(), P, 0, old, P, ref, w, o, P, P, d, ld, None)

    nan, inf = float("nan"), float("inf")
    for kw, code in ((dict(lo=-0.1), 1), (dict(lo=1.1), 1), (dict(lo=nan), 1), (dict(hi=-1.0), 1),
                     (dict(hi=inf), 1), (dict(kl=nan, ref=P), 1), (dict(kl=0.1), 1),
                     (dict(tau=0.0), 1), (dict(d=None), 1), (dict(ld=99), 1), (dict(old=None), 1),
                     (dict(d=P + 2), 3), (dict(w=P + 1), 3), (dict(ref=P + 2), 3),
                     (dict(d=P + 1, z=_z(dtype=1)), 3)):
        assert call(**kw) == code, kw
    assert call(z=_z(rows=0), d=None, old=None) == 0
    assert lib.moe_nvfp4_policy_loss(_z(), P, 0, P, P, None, None, P, P, None) == 1


def test_distill_checks(lib):
    def call(t=None, tau=1.0, out=P, z=None):
        return lib.moe_nvfp4_distill_loss(z or _z(), t or _t(), tau, out, None)

    for t, code in ((_t(K=0), 1), (_t(K=257), 2), (_t(i64=5), 1), (_t(dtype=9), 1),
                    (_t(ids=None), 1), (_t(logits=None), 1), (_t(ids=P + 2), 3),
                    (_t(ids=P + 4, i64=1), 3), (_t(logits=P + 2), 3), (_t(lse=P + 2), 3)):
        assert call(t) == code
    assert call(tau=float("nan")) == 1 and call(out=None) == 1
    assert call(t=_t(ids=None), z=_z(rows=0), out=None) == 0
    assert lib.moe_nvfp4_distill_loss(_z(), None, 1.0, P, None) == 1
    assert lib.moe_nvfp4_distill_loss_grad(_z(), _t(), None, 1.0, P, None, 100, None) == 1


def test_router_checks(lib):
    def batch(z=None, ids=P, mask=None, off=None, K=2, S=1, i64=0, cb=0.01, cz=0.0):
        return M.moe_router_batch(z or _z(cols=8), ids, mask, off, K, S, i64, cb, cz)

    def loss(b, losses=P, ws=P, n=1 << 20):
        return lib.moe_nvfp4_router_loss(b, losses, P, P, ws, n, None)

    for b, code in ((batch(z=_z(cols=1025)), 2), (batch(K=0), 1), (batch(K=9), 2),
                    (batch(z=_z(cols=64), K=33), 2), (batch(S=0), 1), (batch(S=2), 1),
                    (batch(S=(1 << 20) + 1, off=P), 2), (batch(i64=3), 1),
                    (batch(cb=float("nan")), 1), (batch(cz=float("inf")), 1), (batch(ids=None), 1),
                    (batch(ids=P + 2), 3), (batch(off=P + 2), 3),
                    (batch(z=_z(rows=1 << 26, cols=8)), 2)):
        assert loss(b) == code
    assert loss(batch(), losses=None) == 1 and loss(batch(), ws=None) == 1
    assert loss(batch(), ws=P + 16) == 3 and loss(batch(), n=64) == 4

    def grad(b, w=None, dw=None, d=P, ld=8, lg=None):
        return lib.moe_nvfp4_router_loss_grad(b, P, P, lg, w, dw, d, ld, None)

    assert grad(batch(), w=P) == 1 and grad(batch(), dw=P) == 1 and grad(batch(), d=None) == 1
    assert grad(batch(), ld=7) == 1 and grad(batch(), w=P + 2, dw=P) == 3
    assert grad(batch(), lg=P + 2) == 3
    assert grad(batch(z=_z(rows=0, cols=8, data=None))) == 0


def test_router_workspace_sizes(lib):
    size = M.moe_nvfp4_router_loss_workspace_bytes
    for args in ((-1, 8, 1), (4, 0, 1), (4, 1025, 1), (4, 8, 0), (4, 1024, (1 << 20) + 1)):
        assert size(*args) == 0
    prev = 0
    for T in (0, 1, 128, 129, 5000, 1 << 20):
        assert size(T, 256) >= prev > -1
        prev = size(T, 256)
    assert size(100, 64, 10) > size(100, 64, 1)
    with pytest.raises(M.MoeError):
        M.router_loss_workspace(4, 2000, device="cpu")
