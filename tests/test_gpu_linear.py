"""The linear product (moe_linear) and its backward pass against a 64-bit form:
both kernels and the border between them, narrow and ragged outputs, every
epilogue, pitches and alignments, k in parts, gradients against differences."""
import pytest
import torch

import moe_routed_expert_top_b200 as M
from moe_routed_expert_top_b200.layer import Linear
from tests import ops_ref as R
from tests.gpu_util import DEV, ensure_built

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def gen(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, sd=1.0, dt=BF16: torch.empty(*s, dtype=dt, device=DEV).normal_(0, sd, generator=g)


def pitched(t, pitch, shift=0):
    """The same values in rows `pitch` apart, `shift` values behind an aligned address."""
    rows, cols = t.shape
    store = torch.full((rows * pitch + shift + 8,), torch.nan, dtype=t.dtype, device=t.device)
    v = store[shift:].as_strided((rows, cols), (pitch, 1), shift)
    v.copy_(t)
    return v


SHAPES = [(1, 1, 8), (1, 256, 7168), (3, 300, 24), (8, 148, 512), (9, 1200, 1032), (16, 2369, 64), (17, 4736, 264),
          (33, 5000, 136), (63, 37, 2048), (64, 512, 1024), (65, 512, 1024), (65, 1, 8), (100, 6, 4096), (128, 33, 40),
          (129, 255, 264), (256, 256, 128), (257, 257, 136), (300, 1000, 3200), (1000, 64, 72), (2049, 96, 520),
          (700, 3000, 192)]


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)), ids=str)
def test_forward(i, shape):
    m, n, k = shape
    r = gen(i)
    name = ["none", "relu", "silu", "gelu"][i % 4]
    x, w = r(m, k), r(n, k, sd=k ** -0.5)
    bias = [None, r(n, dt=F32), r(n)][i % 3]
    res = [r(m, n), None, r(m, n, dt=F32)][i % 3]
    for out in (BF16, F32):
        L = Linear(w, bias, name, out)
        y, z = L.forward(x, residual=res, with_z=True)
        ref, tol, zr, dz = R.linear(x, w, bias, name, res, out)
        R.check(y, ref, tol, "y")
        R.check(z, zr, dz + R.half(BF16) * (zr.abs() + dz), "z")
        assert L.device_status() == 0
        assert torch.equal(L.forward(x, residual=res), y)  # the same bits without z, and again


@pytest.mark.parametrize("m", [5, 40, 200])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 9), (2, 6), (8, 16)])
def test_pitches_and_alignments(m, shift, pad):
    n, k = 200, 192
    r = gen(m + shift)
    x, w, bias, res = r(m, k), r(n, k, sd=0.1), r(n), r(m, n)
    xp, wp = pitched(x, k + 8 * (1 + pad % 3), 8 * (shift % 2)), pitched(w, k + 16 + 8 * (pad % 2), 8 * (shift % 3))
    rp, yp = pitched(res, n + pad, shift), pitched(torch.zeros_like(res), n + pad + 1, shift)
    L = Linear(wp, bias, "silu")
    y = L.forward(xp, residual=rp, out=yp)
    ref, tol, _, _ = R.linear(x, w, bias, "silu", res, BF16)
    R.check(y, ref, tol)
    gap = yp.as_strided((m - 1, pad + 1), (n + pad + 1, 1), yp.storage_offset() + n)
    assert gap.isnan().all()                               # nothing between the rows was written
    # y may be the residual
    q = pitched(res, n + pad, shift)
    R.check(L.forward(xp, residual=q, out=q), ref, tol)
    # backward with dy, z at such addresses
    z = pitched(r(m, n), n + pad + 3, shift + 1)
    dy = pitched(r(m, n), n + pad, shift)
    got = L.backward(dy, xp, z)
    for g, (a, t) in zip(got, R.linear_backward(dy, x, w, z, "silu")):
        R.check(g, a, t)


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)), ids=str)
def test_backward(i, shape):
    m, n, k = shape
    r = gen(i + 50)
    name = ["gelu", "none", "relu", "silu"][i % 4]
    out = [BF16, F32, BF16][i % 3]
    x, w = r(m, k), r(n, k, sd=k ** -0.5)
    dy, z = r(m, n, dt=out), r(m, n, sd=2.0)
    L = Linear(w, r(n), name, out)
    want = R.linear_backward(dy, x, w, z, name)
    got = L.backward(dy, x, z)
    for what, g, (a, t) in zip(("dx", "dw", "dbias"), got, want):
        R.check(g, a, t, what)
    assert L.device_status() == 0
    # each alone: the same bits are not promised (the parts may be cut otherwise), the tolerance is
    for j in range(3):
        one = L.backward(dy, x, z, *[q == j for q in range(3)])
        assert [v is None for v in one] == [q != j for q in range(3)]
        R.check(one[j], *want[j], f"alone {j}")
    again = L.backward(dy, x, z)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("res_dt", [None, BF16, F32])
@pytest.mark.parametrize("m,n,k,pad", [(300, 773, 200, 0), (257, 289, 1096, 1), (700, 260, 64, 3), (129, 520, 72, 4)])
def test_rows_at_odd_addresses(m, n, k, pad, res_dt, out):
    """Several tiles whose rows begin anywhere, their last columns single: y, z and the
    residual each at another offset, and nothing written beside them."""
    r = gen(m)
    x, w, bias = r(m, k), r(n, k, sd=k ** -0.5), r(n)
    res = None if res_dt is None else pitched(r(m, n, dt=res_dt), n + pad, 1)
    L = Linear(w, bias, "gelu", out)
    yp = pitched(torch.zeros(m, n, dtype=out, device=DEV), n + pad + 1, 3)
    y, z = L.forward(x, residual=res, out=yp, with_z=True)
    ref, tol, zr, dz = R.linear(x, w, bias, "gelu", res, out)
    R.check(y, ref, tol, "y")
    R.check(z, zr, dz + R.half(BF16) * (zr.abs() + dz), "z")
    gap = yp.as_strided((m - 1, pad + 1), (n + pad + 1, 1), yp.storage_offset() + n)
    assert gap.isnan().all()
    if res_dt == out:  # y may be the residual
        R.check(L.forward(x, residual=res, out=res), ref, tol, "in place")


@pytest.mark.parametrize("m", [8, 9, 16])
def test_few_rows_of_a_large_weight(m):
    """With a workspace and without one: the weight on tiles and streamed."""
    n, k = 5001, 8200
    r = gen(m)
    x, w, bias, res = r(m, k), r(n, k, sd=k ** -0.5), r(n), r(m, n)
    ref, tol, _, _ = R.linear(x, w, bias, "silu", res, BF16)
    R.check(Linear(w, bias, "silu").forward(x, residual=res), ref, tol, "layer")
    d = M.make_linear_desc(m, n, k, "silu")
    y = torch.full((m, n), torch.nan, dtype=BF16, device=DEV)
    M.moe_linear(d, x, w, bias, res, y, None)
    R.check(y, ref, tol, "no workspace")


@pytest.mark.parametrize("m,n,k", [(20, 5000, 2056), (1, 4999, 2048), (128, 6001, 1048)])
def test_backward_of_few_rows_and_a_wide_output(m, n, k):
    """dx sums over many columns of y on few tiles, dw has many tiles of one block."""
    r = gen(n)
    x, w, dy = r(m, k), r(n, k, sd=k ** -0.5), r(m, n)
    got = Linear(w, r(n)).backward(dy, x)
    for what, g, (a, t) in zip(("dx", "dw", "dbias"), got, R.linear_backward(dy, x, w, None, "none")):
        R.check(g, a, t, what)


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_gradients_against_differences(name):
    """Inputs whose z is exact in bf16, so that the kernel's formula is that of the
    differentiated function: <gradient, v> against a central difference in 64 bits."""
    m, n, k = 70, 24, 16
    g = torch.Generator(device=DEV).manual_seed(4)
    pick = lambda *s: torch.randint(-1, 2, s, device=DEV, generator=g).double()
    x, w, b = pick(m, k), pick(n, k) / 2, pick(n) / 2      # z: halves up to 8.5, exact
    dy = torch.randn(m, n, device=DEV, generator=g).to(BF16).double()
    z = (x @ w.t() + b).to(BF16)
    assert torch.equal(z.double(), x @ w.t() + b)
    L = Linear(w.to(BF16), b.float(), name)
    got = L.backward(dy.to(BF16), x.to(BF16), z)
    loss = lambda x, w, b: (dy * R.act(x @ w.t() + b, name)).sum()
    for j, (p, grad) in enumerate(zip((x, w, b), got)):
        v = torch.randn(p.shape, device=DEV, generator=g, dtype=torch.float64)
        h = 1e-5
        args = [x, w, b]
        hi, lo = (loss(*[a + s * h * v if q == j else a for q, a in enumerate(args)]) for s in (1, -1))
        ref, tol = R.linear_backward(dy.to(BF16), x, w, z, name)[j]
        diff = (hi - lo) / (2 * h)
        # the difference itself: third derivatives below 4, h^2, and 64-bit noise
        slack = (tol * v.abs()).sum() + 1e-4 * v.abs().sum()
        assert (diff - (grad.double() * v).sum()).abs() <= slack


@pytest.mark.parametrize("name", ["relu", "silu", "gelu"])
def test_activation_far_out(name):
    """Tails, infinities and NaN: x = 1, w = the value."""
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, -13.0, 20.0, -20.0, 90.0, -90.0, 3e38, -3e38, torch.inf,
                      torch.nan], device=DEV).to(BF16)
    w = torch.zeros(v.numel(), 8, dtype=BF16, device=DEV)
    w[:, 0] = v
    z = v.double()
    want = R.act(z, name)
    for m in (2, 70):
        x = torch.zeros(m, 8, dtype=BF16, device=DEV)
        x[:, 0] = 1
        y = Linear(w, None, name, F32).forward(x).double()
        dy = torch.ones(m, v.numel(), device=DEV)
        db = Linear(w, torch.zeros(v.numel(), device=DEV), name, F32).backward(dy, x, v.expand(m, -1).contiguous(),
                                                                                False, False)[2].double() / m
        for got, ref in ((y[0], want), (db, R.slope(z, name))):
            fin = ref.isfinite() & z.isfinite()
            # float has no value below 1e-38: what underflows there is 0
            assert ((got - ref).abs()[fin] <= 1e-5 * ref.abs()[fin] + 1e-37).all(), (name, got, ref)
        assert y[0][-1].isnan() and y[0][-2] == torch.inf


def test_row_border_and_empty():
    r = gen(1)
    w = r(96, 64)
    L = Linear(w, r(96), "gelu")
    e = L.forward(torch.empty(0, 64, dtype=BF16, device=DEV))
    assert e.shape == (0, 96)
    dx, dw, db = L.backward(torch.empty(0, 96, dtype=BF16, device=DEV), torch.empty(0, 64, dtype=BF16, device=DEV),
                            torch.empty(0, 96, dtype=BF16, device=DEV))
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    n0 = Linear(torch.empty(0, 64, dtype=BF16, device=DEV))
    assert n0.forward(r(3, 64)).shape == (3, 0)
    dx, dw, _ = n0.backward(torch.empty(3, 0, dtype=BF16, device=DEV), r(3, 64))
    assert (dx == 0).all() and dw.shape == (0, 64)


def test_rows_past_32_bit_offsets():
    """x and y in rows 2**30 values apart."""
    m, n, k = 3, 40, 64
    r = gen(2)
    ld = 2 ** 30 + 16
    store = torch.empty(64 * (2 ** 25 + 8) + 64, dtype=BF16, device=DEV)  # (more than 2 * ld + 64)
    x = store.as_strided((m, k), (ld, 1))
    x.copy_(r(m, k))
    ys = torch.empty((m - 1) * ld + 64, dtype=BF16, device=DEV)
    y = ys.as_strided((m, n), (ld, 1))
    w = r(n, k)
    Linear(w).forward(x, out=y)
    ref, tol, _, _ = R.linear(x, w, None, "none", None, BF16)
    R.check(y, ref, tol)
    del ys, y
    torch.cuda.empty_cache()
    big = store.as_strided((65, k), (2 ** 25 + 8, 1))       # the tiled kernel, 2.2e9 values of span
    big.copy_(r(65, k))
    ref, tol, _, _ = R.linear(big, w, None, "none", None, BF16)
    R.check(Linear(w).forward(big), ref, tol)


def test_streams_and_graphs():
    r = gen(3)
    x, w, dy, z = r(200, 512), r(320, 512, sd=0.05), r(200, 320), r(200, 320)
    L = Linear(w, r(320), "silu")
    want = [L.forward(x), *L.backward(dy, x, z)]
    torch.cuda.synchronize()
    outs = []
    for st in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(st):
            outs.append([L.forward(x), *L.backward(dy, x, z)])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(g):
        cap = [L.forward(xs), *L.backward(dy, xs, z)]
    xs.copy_(r(200, 512))
    g.replay()
    xs.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    for o in outs + [cap]:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_python_checks():
    r = gen(4)
    L = Linear(r(32, 64), None, "relu")
    for bad in (lambda: L.forward(r(4, 72)), lambda: L.forward(r(4, 64, dt=F32)), lambda: L.forward(r(64, 4).t()),
                lambda: L.forward(r(4, 64).cpu()), lambda: L.forward(r(4, 64), residual=r(4, 31)),
                lambda: L.backward(r(4, 32), r(4, 64)), lambda: Linear(r(3, 4), activation="tanh"),
                lambda: Linear(r(3, 8), r(4)), lambda: Linear(r(3, 8), out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(M.MoeError):                        # K % 8
        Linear(r(32, 60)).forward(r(4, 60))
