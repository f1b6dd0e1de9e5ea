"""64-bit forms of the few-token layer, the linear product and layer norm, and how
far a kernel's result may be from them.

Tolerances count roundings. A value rounded once to type t is off by at most
`half(t)` of itself; an fp32 sum of n products is off by at most n steps of 2**-23 of
the sum of their magnitudes (the tensor core drops bits, so a whole step for each
addition and not half a one); the fast exponential and division of the
activations and the fitted normal distribution function are good to 2**-18."""
from __future__ import annotations

import torch

STEP = 2.0 ** -23
FAST = 2.0 ** -18


def half(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z * 0.5 ** 0.5)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(-z * 0.5 ** 0.5) + z * torch.exp(-0.5 * z * z) * (0.5 / torch.pi) ** 0.5
    return torch.ones_like(z)


def expert(x, w_gate_up, w_down):
    """(rows [n, H] through one expert, how far an fp32 kernel that rounds h to bf16 may be)."""
    F = w_down.shape[1]
    x, wu, wd = x.double(), w_gate_up.double(), w_down.double()
    both, size = x @ wu.t(), x.abs() @ wu.abs().t()
    g, u = both[:, :F], both[:, F:]
    dg, du = x.shape[1] * STEP * size[:, :F], x.shape[1] * STEP * size[:, F:]
    sg = act(g, "silu")
    h = sg * u
    dh = 1.1 * dg * u.abs() + (sg.abs() + 1.1 * dg) * du + FAST * h.abs()
    dh = dh + half(torch.bfloat16) * (h.abs() + dh)
    y = h @ wd.t()
    return y, dh @ wd.abs().t() + F * STEP * ((h.abs() + dh) @ wd.abs().t())


def layer(x, ids, weights, w_gate_up, w_down, scale, ws_gate_up=None, ws_down=None, residual=None):
    """(out [T, H], tolerance) of the routed layer; ids outside [0, E) are skipped."""
    T, E = x.shape[0], w_gate_up.shape[0]
    out = torch.zeros(T, x.shape[1], dtype=torch.float64, device=x.device)
    tol, size = torch.zeros_like(out), torch.zeros_like(out)
    for e in sorted(set(int(i) for i in ids.flatten().tolist()) & set(range(E))):
        hit = ids == e
        rows = hit.any(1).nonzero()[:, 0]
        y, dy = expert(x[rows], w_gate_up[e], w_down[e])
        p = scale * (weights.double() * hit)[rows].sum(1, keepdim=True)
        out[rows] += p * y
        tol[rows] += p.abs() * dy
        size[rows] += (p * y).abs()
    if ws_gate_up is not None:
        y, dy = expert(x, ws_gate_up, ws_down)
        out, tol, size = out + y, tol + dy, size + y.abs()
    if residual is not None:
        out, size = out + residual.double(), size + residual.double().abs()
    terms = ids.shape[1] + 12  # additions of whole terms, and of the warps' parts
    tol = tol + terms * STEP * size
    return out, tol + half(torch.bfloat16) * (out.abs() + tol)


def linear(x, w, bias, name, residual, out):
    """(y, tolerance, z, tolerance of z before its rounding)."""
    x, w = x.double(), w.double()
    z, dz = x @ w.t(), (x.shape[1] + 16) * STEP * (x.abs() @ w.abs().t())
    if bias is not None:
        z = z + bias.double()
        dz = dz + STEP * z.abs()
    a = act(z, name)
    y, tol = a, 1.13 * dz + FAST * a.abs()
    if residual is not None:
        y = y + residual.double()
        tol = tol + STEP * (a.abs() + residual.double().abs())
    return y, tol + half(out) * (y.abs() + tol), z, dz


def linear_backward(dy, x, w, z, name):
    """((dx, tolerance), (dw, tolerance), (dbias, tolerance)); z as the kernel gets it."""
    d, x, w = dy.double(), x.double(), w.double()
    bf16 = half(torch.bfloat16)
    dd = torch.zeros_like(d)
    rounded = dy.dtype != torch.bfloat16
    if name != "none":
        s = slope(z.double(), name)
        # silu'(z) and gelu'(z) are sums of terms up to 1.5 in size
        dd = d.abs() * (FAST * 1.5) + STEP * d.abs() * s.abs()
        d = d * s
        rounded = True
    op = dd + (bf16 * (d.abs() + dd) if rounded else 0)  # the products' operand
    out = []
    for a, b, n, size in ((d @ w, (d.abs() + op) @ w.abs(), w.shape[0], op @ w.abs()),
                          (d.t() @ x, (d.abs() + op).t() @ x.abs(), x.shape[0], op.t() @ x.abs())):
        tol = size + (n + 16) * STEP * b
        out.append((a, tol + bf16 * (a.abs() + tol)))
    db = d.sum(0)
    out.append((db, dd.sum(0) + (x.shape[0] + 64) * STEP * d.abs().sum(0)))
    return out


def norm(x, gamma, beta, eps):
    """((y, tolerance), (mean, tolerance), (rstd, tolerance))."""
    t, H = x.dtype, x.shape[1]
    x = x.double()
    g = torch.ones(H, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    b = torch.zeros(H, dtype=torch.float64, device=x.device) if beta is None else beta.double()
    n = 64 + H / 256  # additions in a chain: a thread's values, then the tree over the threads
    mean = x.mean(1)
    dm = n * STEP * x.abs().mean(1) + STEP * mean.abs()
    far = x - mean[:, None]
    var = (far * far).mean(1)
    # |far| is off by dm + a rounding of it
    df = dm[:, None] + STEP * far.abs()
    dv = (2 * far.abs() * df + df * df).mean(1) + (n + 4) * STEP * var
    rstd = (var + eps) ** -0.5
    low = (var + eps - dv - STEP * (var + eps)).clamp_min(0)
    dr = torch.where(low > 0, low.clamp_min(1e-300) ** -0.5 - rstd, torch.inf * rstd) + 4 * STEP * rstd
    y = far * rstd[:, None] * g + b
    tol = (df * rstd[:, None] + (far.abs() + df) * dr[:, None]) * g.abs() + 4 * STEP * (
        (far * rstd[:, None] * g).abs() + b.abs())
    return (y, tol + half(t) * (y.abs() + tol)), (mean, dm), (rstd, dr)


def norm_backward(dy, x, gamma, mean, rstd):
    """((dx, tolerance), (dgamma, tolerance), (dbeta, tolerance)); mean, rstd as the kernel gets them."""
    t, (M, H) = x.dtype, x.shape
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    g = torch.ones(H, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    far = x - mean
    xh = far * rstd
    dxh = 2 * STEP * xh.abs()
    gg = dy * g
    n = 64 + H / 256
    c1, c2 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    d1 = (n + 2) * STEP * gg.abs().mean(1, keepdim=True)
    d2 = (n + 4) * STEP * (gg * xh).abs().mean(1, keepdim=True)
    dx = rstd * (gg - c1 - xh * c2)
    size = gg.abs() + c1.abs() + (xh * c2).abs()
    tol = rstd * (d1 + xh.abs() * d2 + dxh * c2.abs() + 6 * STEP * size)
    m = 64 + M / 64
    dgam, dbet = (dy * xh).sum(0), dy.sum(0)
    return ((dx, tol + half(t) * (dx.abs() + tol)),
            (dgam, (m + 4) * STEP * (dy * xh).abs().sum(0)), (dbet, m * STEP * dy.abs().sum(0)))


def check(got, ref, tol, what=""):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = (got - ref).abs()
    bad = ~(err <= tol) & ~(got == ref) & ~(got.isnan() & ref.isnan())
    if bad.any():
        i = torch.where(bad, err - tol, torch.full_like(err, -1.0)).nan_to_num(torch.inf).argmax()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; at {int(i)}: got "
                             f"{got.flatten()[i].item()!r} ref {ref.flatten()[i].item()!r} tolerance "
                             f"{tol.flatten()[i].item():.3e}")
