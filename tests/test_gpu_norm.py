"""Layer norm and its backward pass against a 64-bit form: row lengths on both
sides of every kernel's border, odd lengths, pitches and addresses, both types."""
import pytest
import torch

from moe_routed_expert_top_b200.layer import LayerNorm
from tests import ops_ref as R
from tests.gpu_util import DEV, ensure_built

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def gen(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, sd=1.0, mean=0.0, dt=BF16: torch.empty(*s, dtype=dt, device=DEV).normal_(mean, sd, generator=g)


def pitched(t, pitch, shift):
    rows, cols = t.shape
    store = torch.full((max(rows - 1, 0) * pitch + cols + shift,), torch.nan, dtype=t.dtype, device=t.device)
    v = store.as_strided((rows, cols), (pitch, 1), shift)
    v.copy_(t)
    return v


def both_ways(x, w, b, dy, eps=1e-5, out=None):
    L = LayerNorm(w, b, eps)
    y, mean, rstd = L.forward(x, out=out, stats=True)
    for what, got, (ref, tol) in zip(("y", "mean", "rstd"), (y, mean, rstd), R.norm(x, w, b, eps)):
        R.check(got, ref, tol, what)
    got = L.backward(dy, x, mean, rstd)
    for what, g, (ref, tol) in zip(("dx", "dgamma", "dbeta"), got, R.norm_backward(dy, x, w, mean, rstd)):
        R.check(g, ref, tol, what)
    assert torch.equal(L.forward(x), y)                    # without the statistics, and again
    assert all(torch.equal(a, c) for a, c in zip(L.backward(dy, x, mean, rstd), got))
    return y, mean, rstd, got


LENGTHS = [1, 2, 3, 7, 8, 16, 31, 33, 255, 512, 513, 1000, 1023, 1024, 1025, 1026, 2047, 2048, 2050, 4097, 7168, 8191,
           8192, 8193, 8200, 12288, 16383, 16384, 16385, 20000]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", LENGTHS)
def test_lengths(H, dt):
    r = gen(H)
    wdt = F32 if H % 3 == 0 else dt
    for m in (1, 5, 700):
        w, b = r(H, sd=0.2, mean=1.0, dt=wdt), r(H, sd=0.2, dt=wdt)
        both_ways(r(m, H, sd=2.0, mean=0.5, dt=dt), w, b, r(m, H, dt=dt))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,pad,shift", [(64, 8, 0), (100, 4, 2), (1000, 1, 1), (1536, 3, 5), (2048, 16, 8), (2049, 0, 3),
                                         (2050, 2, 6), (4096, 5, 1), (9000, 7, 3), (17000, 1, 1)])
def test_pitches_and_addresses(H, pad, shift, dt):
    r = gen(H + pad)
    w, b = r(H + 1, dt=dt)[1:], r(H + 3, dt=dt)[3:]        # views: the object keeps them as they are
    for m in (1, 2, 37):
        x, dy = pitched(r(m, H, dt=dt), H + pad, shift), pitched(r(m, H, dt=dt), H + pad + 1, shift + 1)
        out = pitched(torch.zeros(m, H, dtype=dt, device=DEV), H + pad + 2, shift)
        both_ways(x, w, b, dy, out=out)
        if m > 1:
            gap = out.as_strided((m - 1, pad + 2), (H + pad + 2, 1), out.storage_offset() + H)
            assert gap.isnan().all()


@pytest.mark.parametrize("H", [48, 3000])
def test_without_weights_and_parts(H):
    r = gen(1)
    x, dy, w, b = r(33, H), r(33, H), r(H), r(H)
    both_ways(x, None, None, dy)
    both_ways(x, w, None, dy)
    both_ways(x, None, b, dy)
    L = LayerNorm(w, b)
    _, mean, rstd = L.forward(x, stats=True)
    whole = L.backward(dy, x, mean, rstd)
    dx, dw, db = L.backward(dy, x, mean, rstd, need_weights=False)
    assert dw is None and db is None and torch.equal(dx, whole[0])
    dx, dw, db = L.backward(dy, x, mean, rstd, need_dx=False)
    assert dx is None and torch.equal(dw, whole[1]) and torch.equal(db, whole[2])


@pytest.mark.parametrize("H", [40, 2304, 20480])
def test_in_place(H):
    import moe_routed_expert_top_b200 as M
    r = gen(2)
    m = 300
    x, dy, w, b = r(m, H), r(m, H), r(H), r(H)
    L = LayerNorm(w, b)
    want, mean, rstd = L.forward(x, stats=True)
    q = x.clone()
    assert torch.equal(L.forward(q, out=q), want)
    grads = L.backward(dy, x, mean, rstd)
    for which in (0, 1):                                   # dx in dy's place, in x's
        a = [dy.clone(), x.clone()]
        dg, db = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
        ws = torch.empty(M.moe_layer_norm_backward_workspace_bytes(m, H), dtype=torch.uint8, device=DEV)
        M.moe_layer_norm_backward(m, H, 0, 0, 0, False, False, a[0], a[1], w, mean, rstd, a[which], dg, db, ws)
        for got, ref in zip((a[which], dg, db), grads):
            assert torch.equal(got, ref)


def test_rows_that_are_hard():
    """A large common offset, a constant row, a row of zeros, one outlier, values near
    the type's end."""
    H = 2304
    r = gen(3)
    for dt in (BF16, F32):
        x = r(6, H, dt=dt)
        x[0] = (x[0].float() + 1000.0).to(dt)
        x[1] = 3.0
        x[2] = 0.0
        x[3, 77] = 1e4
        x[4] *= 1e-15
        x[5] *= 1e15
        both_ways(x, r(H, dt=dt), r(H, dt=dt), r(6, H, dt=dt))


def test_infinities_and_nan_stay_in_their_row():
    H = 3000
    r = gen(4)
    x, dy, w = r(5, H), r(5, H), r(H)
    x[1, 5], x[3, 2999] = torch.inf, torch.nan
    L = LayerNorm(w, None)
    y, mean, rstd = L.forward(x, stats=True)
    good = [0, 2, 4]
    assert y[[1, 3]].isnan().all() and y[good].isfinite().all()
    dx, _, _ = L.backward(dy, x, mean, rstd)
    assert dx[[1, 3]].isnan().all() and dx[good].isfinite().all()


def test_differences():
    """<gradient, v> against a central difference of the 64-bit function."""
    m, H, eps = 6, 50, 1e-3
    g = torch.Generator(device=DEV).manual_seed(5)
    x, dy = (torch.randn(m, H, device=DEV, generator=g) for _ in range(2))
    w, b = (torch.randn(H, device=DEV, generator=g) for _ in range(2))
    L = LayerNorm(w, b, eps)
    _, mean, rstd = L.forward(x, stats=True)
    got = L.backward(dy, x, mean, rstd)
    tols = [t for _, t in R.norm_backward(dy, x, w, mean, rstd)]
    f = lambda x, w, b: (dy.double() * torch.nn.functional.layer_norm(x, (H,), w, b, eps)).sum()
    args = [x.double(), w.double(), b.double()]
    for j in range(3):
        v = torch.randn(args[j].shape, device=DEV, generator=g, dtype=torch.float64)
        h = 1e-5
        hi, lo = (f(*[a + s * h * v if q == j else a for q, a in enumerate(args)]) for s in (1, -1))
        # mean and rstd reach the kernel rounded: 2**-22 of the terms they enter
        slack = (tols[j] * v.abs()).sum() + 2.0 ** -20 * (got[j].double().abs() * v.abs()).sum() + 1e-5 * v.abs().sum()
        assert ((hi - lo) / (2 * h) - (got[j].double() * v).sum()).abs() <= slack


def test_empty_rows_offsets_streams_graph():
    r = gen(6)
    w, b = r(64), r(64)
    L = LayerNorm(w, b)
    e = torch.empty(0, 64, dtype=BF16, device=DEV)
    y, mean, rstd = L.forward(e, stats=True)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = L.backward(e, e, mean, rstd)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    ld = 2 ** 30 + 8
    store = torch.empty(2 * ld + 64, dtype=BF16, device=DEV)
    x = store.as_strided((3, 64), (ld, 1))
    x.copy_(r(3, 64))
    both_ways(x, w, b, r(3, 64))
    del store, x
    x, dy = r(500, 2048), r(500, 2048)
    L = LayerNorm(r(2048), r(2048))
    y, mean, rstd = L.forward(x, stats=True)
    want = [y, *L.backward(dy, x, mean, rstd)]
    torch.cuda.synchronize()
    outs = []
    for st in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(st):
            outs.append([L.forward(x), *L.backward(dy, x, mean, rstd)])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        yc, m2, r2 = L.forward(x, stats=True)
        cap = [yc, *L.backward(dy, x, m2, r2)]
    g.replay()
    torch.cuda.synchronize()
    for o in outs + [cap]:
        assert all(torch.equal(a, c) for a, c in zip(o, want))


def test_python_checks():
    r = gen(7)
    L = LayerNorm(r(64), r(64))
    x = r(4, 64)
    _, mean, rstd = L.forward(x, stats=True)
    for bad in (lambda: L.forward(r(4, 65)), lambda: L.forward(r(64, 4).t()), lambda: L.forward(x.to(torch.float16)),
                lambda: L.forward(x, out=torch.empty(4, 64, device=DEV)), lambda: L.backward(r(4, 64, dt=F32), x, mean, rstd),
                lambda: L.backward(x, x, mean[:3], rstd), lambda: LayerNorm(r(64), r(64, dt=F32)),
                lambda: LayerNorm(r(64), eps=-1.0), lambda: LayerNorm(r(64), eps=float("nan"))):
        with pytest.raises(ValueError):
            bad()
