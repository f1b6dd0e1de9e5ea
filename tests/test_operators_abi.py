"""Host-side checks of the few-token layer, the linear product and layer norm (no
GPU needed: nothing here launches a kernel)."""
import ctypes

import pytest

F = ctypes.c_float
Z = ctypes.c_size_t
BIG = Z(1 << 40)


@pytest.fixture(scope="module")
def M():
    from moe_routed_expert_top_b200 import build
    build.build()
    import moe_routed_expert_top_b200 as m
    return m


def few(M, hidden=32, logits=32, ids=None, w=None, gu=32, dn=32, sgu=None, sd=None, res=None, out=32, ws=32, n=BIG,
        **kw):
    p = M.make_problem(**{**dict(T=4, H=256, F=128, E=8, top_k=2), **kw})
    return M.lib().moe_experts_forward_few(ctypes.byref(p), hidden, logits, ids, w, gu, dn, sgu, sd, F(1.0), res, out,
                                           ws, n, None)


def test_few_refusals(M):
    L = M.lib()
    assert few(M, T=0, hidden=None, out=None, ws=None) == 0
    for kw, status in ((dict(T=65), -2), (dict(T=-1), -1), (dict(down_fp8=True, F=128), -2), (dict(H=96), -2),
                       (dict(F=100), -2), (dict(E=1025), -2), (dict(top_k=9), -2), (dict(top_k=0), -1),
                       (dict(padding_M=64), -2), (dict(score_fn=5), -1), (dict(F_shared=64), -1),
                       (dict(F_shared=100), -2)):
        assert few(M, **kw) == status, kw
    for kw in (dict(hidden=None), dict(gu=None), dict(dn=None), dict(out=None), dict(ws=None), dict(logits=None),
               dict(logits=None, ids=32), dict(hidden=40), dict(gu=48), dict(dn=16), dict(out=8), dict(res=8),
               dict(ws=8), dict(logits=34), dict(ids=33), dict(F_shared=64, sgu=32), dict(F_shared=64, sgu=48, sd=32)):
        assert few(M, **kw) == -1, kw
    need = M.moe_few_workspace_bytes(M.make_problem(T=4, H=256, F=128, E=8, top_k=2))
    assert need >= 4 * 2 * 128 * 2 + 1024
    assert few(M, n=Z(need - 1)) == -3
    assert M.moe_few_workspace_bytes(M.make_problem(T=65, H=256, F=128, E=8, top_k=2)) == 0
    assert L.moe_experts_forward_few(None, 32, 32, None, None, 32, 32, None, None, F(1.0), None, 32, 32, BIG,
                                     None) == -1


def linear(mod, x=32, w=32, b=None, r=None, y=32, z=None, ws=32, n=BIG, **kw):
    d = mod.make_linear_desc(**{**dict(M=4, N=16, K=64), **kw})
    return mod.lib().moe_linear(ctypes.byref(d), x, w, b, r, y, z, ws, n, None)


def linear_bwd(mod, dy=32, x=32, w=32, z=None, dx=32, dw=32, db=None, ws=32, n=BIG, **kw):
    d = mod.make_linear_desc(**{**dict(M=4, N=16, K=64), **kw})
    return mod.lib().moe_linear_backward(ctypes.byref(d), dy, x, w, z, dx, dw, db, ws, n, None)


def test_linear_refusals(M):
    L = M.lib()
    assert linear(M, M=0, x=None, y=None, ws=None) == 0
    assert linear(M, N=0, x=None, y=None, ws=None) == 0
    for f in (linear, linear_bwd):
        for kw, status in ((dict(M=-1), -1), (dict(N=-1), -1), (dict(K=0), -1), (dict(K=60), -2), (dict(act=4), -1),
                           (dict(act=-1), -1), (dict(ldx=63), -1), (dict(ldx=68), -2), (dict(ldw=56), -1),
                           (dict(ldw=65), -2), (dict(ldy=15), -1), (dict(ldz=15), -1), (dict(ldr=15), -1),
                           (dict(ldx=-64), -1), (dict(M=(1 << 24) + 1), -2), (dict(K=1 << 25), -2),
                           (dict(ldx=1 << 40), -2), (dict(x=40), -1), (dict(w=40), -1), (dict(ws=16), -1),
                           (dict(M=65, ws=None), -1), (dict(z=33), -1)):
            assert f(M, **kw) == status, (f.__name__, kw)
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(b=33), dict(b=34, bias_f32=True), dict(r=33),
               dict(r=34, res_f32=True), dict(y=33), dict(y=34, y_f32=True)):
        assert linear(M, **kw) == -1, kw
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(ws=None), dict(act="silu"), dict(dy=33), dict(dy=34, y_f32=True),
               dict(dx=40), dict(dw=40), dict(db=34)):
        assert linear_bwd(M, **kw) == -1, kw
    d = M.make_linear_desc(M=4, N=16, K=64)
    d.reserved = 1
    assert L.moe_linear(ctypes.byref(d), 32, 32, None, None, 32, None, 32, BIG, None) == -1
    assert L.moe_linear(None, 32, 32, None, None, 32, None, 32, BIG, None) == -1
    assert linear(M, n=Z(1023)) == -3
    assert linear_bwd(M, n=Z(1023)) == -3
    assert linear_bwd(M, dx=None, dw=None, db=None, dy=None, ws=None) == 0


@pytest.mark.parametrize("m,n,k,f32", [(1, 1, 8, 0), (64, 100, 64, 1), (65, 100, 64, 0), (300, 7, 8192, 1),
                                       (4096, 7168, 2048, 0), (100, 256, 1 << 20, 1), (1 << 24, 8, 8, 0)])
def test_linear_workspace(M, m, n, k, f32):
    d = M.make_linear_desc(m, n, k, y_f32=f32)
    fwd, bwd = M.moe_linear_workspace_bytes(d), M.moe_linear_backward_workspace_bytes(d)
    assert fwd >= 1024 and bwd >= 1024 + m * ((n + 7) // 8 * 8) * 2
    parts = (k + 2047) // 2048
    if f32 and m > 64 and parts > 1:                       # an fp32 result comes in parts of 2048 k
        assert fwd >= 1024 + parts * m * n * 4
    assert M.moe_linear_workspace_bytes(M.make_linear_desc(m, n, 60)) == 0


def test_norm_refusals(M):
    L = M.lib()

    def fwd(m=4, h=64, ldx=0, ldy=0, xf=0, wf=0, x=32, g=32, b=32, eps=1e-5, y=32, mean=32, rstd=32):
        return L.moe_layer_norm(m, h, ldx, ldy, xf, wf, x, g, b, F(eps), y, mean, rstd, None)

    def bwd(m=4, h=64, lddy=0, ldx=0, lddx=0, xf=0, wf=0, dy=32, x=32, g=32, mean=32, rstd=32, dx=32, dg=32, db=32,
            ws=32, n=BIG):
        return L.moe_layer_norm_backward(m, h, lddy, ldx, lddx, xf, wf, dy, x, g, mean, rstd, dx, dg, db, ws, n, None)

    assert fwd(m=0, x=None, y=None) == 0
    for kw, status in ((dict(m=-1), -1), (dict(h=0), -1), (dict(h=(1 << 24) + 1), -2), (dict(ldx=63), -1),
                       (dict(ldy=63), -1), (dict(ldx=-64), -1), (dict(x=None), -1), (dict(y=None), -1), (dict(x=33), -1),
                       (dict(x=34, xf=1), -1), (dict(g=34, wf=1), -1), (dict(b=33), -1), (dict(mean=34), -1),
                       (dict(rstd=33), -1), (dict(eps=-1e-9), -1), (dict(eps=float("nan")), -1)):
        assert fwd(**kw) == status, kw
    for kw, status in ((dict(m=-1), -1), (dict(h=0), -1), (dict(h=1 << 25), -2), (dict(lddy=3), -1), (dict(lddx=3), -1),
                       (dict(dy=None), -1), (dict(x=None), -1), (dict(mean=None), -1), (dict(rstd=None), -1),
                       (dict(ws=None), -1), (dict(ws=16), -1), (dict(dx=33), -1), (dict(dg=34), -1),
                       (dict(n=Z(16)), -3)):
        assert bwd(**kw) == status, kw
    assert bwd(dx=None, dg=None, db=None, dy=None) == 0
    assert M.moe_layer_norm_backward_workspace_bytes(-1, 4) == 0
    assert M.moe_layer_norm_backward_workspace_bytes(4, 0) == 0
    for m, h in ((1, 1), (4096, 7168), (3, 20000), (1 << 20, 5)):
        assert M.moe_layer_norm_backward_workspace_bytes(m, h) >= 8 * h
