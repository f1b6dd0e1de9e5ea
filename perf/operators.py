"""Cases of three operators that stand around the routed experts of a feed-forward block, and what each computes.

  few          a whole routed mixture-of-experts layer for a few tokens: routing from logits, gate+up, SiLU(gate)*up, down,
               the weighted sum over the experts, the shared expert and the residual
  linear       a matrix product with bias, activation and residual in its epilogue (the router, a dense projection)
  linear_bwd   its backward pass: gradients of the input, the weight and the bias
  norm         layer norm's forward pass, with the row statistics that its backward pass reads
  norm_bwd     layer norm's backward pass: gradients of the input, the weight and the bias

`own` false: elementary torch operations in 32 bits. `own` true: the calls of the framework's operators.
"""
import torch

own = False


def listed():
    return [
        # one token of a decode step, 128 small experts: 75 MB of weights, latency counts
        dict(name="few_1_small", kind="few", T=1, E=128, k=8, H=2048, F=768, Fs=0, score="softmax", residual=True),
        # a ragged decode batch on the same experts
        dict(name="few_13_small", kind="few", T=13, E=128, k=8, H=2048, F=768, Fs=0, score="softmax", residual=False),
        # a few sequences decoded together on large experts, with a shared expert
        dict(name="few_5_large", kind="few", T=5, E=256, k=8, H=7168, F=2048, Fs=2048, score="sigmoid", residual=True),
        # the largest batch of this form: most experts are touched
        dict(name="few_64_large", kind="few", T=64, E=256, k=8, H=7168, F=2048, Fs=2048, score="sigmoid", residual=True),
        # the router's product for one token: fp32 logits from a small weight
        dict(name="linear_router_1", kind="linear", M=1, N=256, K=7168, act="none", bias=True, res=False, f32=True),
        # a dense projection for a ragged decode batch: the weight's bytes decide
        dict(name="linear_17", kind="linear", M=17, N=4608, K=2048, act="gelu", bias=True, res=True, f32=False),
        # a dense projection of a prefill
        dict(name="linear_4096", kind="linear", M=4096, N=7168, K=2048, act="silu", bias=True, res=True, f32=False),
        # the router's backward pass over a ragged batch: fp32 gradients of the logits, a narrow weight
        dict(name="linear_bwd_router", kind="linear_bwd", M=1999, N=256, K=2048, act="none", bias=True, f32=True),
        # a dense projection's backward pass over a training batch
        dict(name="linear_bwd_4096", kind="linear_bwd", M=4096, N=4096, K=7168, act="gelu", bias=True, f32=False),
        # the norm of one decode step
        dict(name="norm_8", kind="norm", M=8, H=7168, f32=False),
        # the norm of a long prefill, rows of an odd size in 32 bits
        dict(name="norm_16383_f32", kind="norm", M=16383, H=2050, f32=True),
        # the norm's backward pass over a training batch
        dict(name="norm_bwd_8192", kind="norm_bwd", M=8192, H=7168, f32=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["few", "few", "linear", "linear_bwd", "norm", "norm_bwd"])
    if kind == "few":
        E = _log(rng, 4, 256)
        return dict(kind=kind, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(8, E)), H=64 * _log(rng, 2, 112),
                    F=64 * _log(rng, 1, 32), Fs=64 * rng.choice([0, 0, _log(rng, 1, 32)]),
                    score=rng.choice(["softmax", "sigmoid"]), residual=rng.random() < 0.5)
    if kind == "linear":
        return dict(kind=kind, M=_log(rng, 1, 4096), N=_log(rng, 1, 7168), K=8 * _log(rng, 4, 896),
                    act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.7, res=rng.random() < 0.5,
                    f32=rng.random() < 0.3)
    if kind == "linear_bwd":
        return dict(kind=kind, M=_log(rng, 1, 4096), N=_log(rng, 1, 4096), K=8 * _log(rng, 4, 896),
                    act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.7, f32=rng.random() < 0.3)
    return dict(kind=kind, M=_log(rng, 1, 8192), H=_log(rng, 1, 8192), f32=rng.random() < 0.4)


def _with_layer(s):
    """The layer object that a program keeps beside its weights: it holds references to them."""
    if own:
        from moe_routed_expert_top_b200 import layer
        case = s["case"]
        if case["kind"] == "few":
            s["layer"] = layer.FewTokenExperts(s["w_gate_up"], s["w_down"], case["k"], case["score"], True, s["scale"],
                                               s["ws_gate_up"], s["ws_down"])
        elif case["kind"] in ("linear", "linear_bwd"):
            s["layer"] = layer.Linear(s["w"], s["bias"], case["act"], torch.float32 if case["f32"] else torch.bfloat16)
        else:
            s["layer"] = layer.LayerNorm(s["w"], s["b"], s["eps"])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)

    s = dict(case=case)
    if kind == "few":
        T, E, H, F, Fs = (case[n] for n in ("T", "E", "H", "F", "Fs"))
        s["x"] = normal(T, H)
        s["logits"] = normal(T, E, dtype=torch.float32)
        s["w_gate_up"] = normal(E, 2 * F, H, std=0.02)
        s["w_down"] = normal(E, H, F, std=0.02)
        s["ws_gate_up"] = normal(2 * Fs, H, std=0.02) if Fs else None
        s["ws_down"] = normal(H, Fs, std=0.02) if Fs else None
        s["residual"] = normal(T, H) if case["residual"] else None
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        return _with_layer(s)
    if kind in ("linear", "linear_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        out = torch.float32 if case["f32"] else torch.bfloat16
        s["x"] = normal(M, K)
        s["w"] = normal(N, K, std=K ** -0.5)
        s["bias"] = normal(N, std=0.5, dtype=torch.float32) if case["bias"] else None
        if kind == "linear":
            s["residual"] = normal(M, N) if case["res"] else None
        else:
            s["dy"] = normal(M, N, dtype=out)
            # what the forward pass keeps: the product with its bias, before the activation
            s["z"] = normal(M, N) if case["act"] != "none" else None
        return _with_layer(s)
    M, H = case["M"], case["H"]
    kept = torch.float32 if case["f32"] else torch.bfloat16
    s["x"] = normal(M, H, std=1.5, mean=0.25, dtype=kept)
    s["w"] = normal(H, std=0.1, mean=1.0, dtype=kept)
    s["b"] = normal(H, std=0.1, dtype=kept)
    s["eps"] = 1e-5
    if kind == "norm_bwd":
        s["dy"] = normal(M, H, dtype=kept)
        # the statistics that the forward pass keeps
        x = s["x"].double()
        s["mean"] = x.mean(1).float()
        s["rstd"] = (1.0 / (x.var(1, unbiased=False) + s["eps"]).sqrt()).float()
    return _with_layer(s)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return z


def _slope(z, act):
    """The derivative of the activation at z."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 / torch.pi) ** 0.5


def _mlp(x, gate_up, down):
    """Rows x [n, H] through experts gate_up [n, 2F, H] and down [n, H, F], one each, in 32 bits."""
    both = torch.bmm(gate_up.float(), x[:, :, None])[:, :, 0]
    half = both.shape[1] // 2
    return torch.bmm(down.float(), (_act(both[:, :half], "silu") * both[:, half:])[:, :, None])[:, :, 0]


def _plain_few(s):
    x, logits, k = s["x"].float(), s["logits"], s["case"]["k"]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    score = torch.exp(top - top[:, :1]) if s["case"]["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-top))
    weight = s["scale"] * score / score.sum(1, keepdim=True)
    out = torch.empty_like(x)
    for t in range(x.shape[0]):  # the experts of one token at a time: all of them together would not fit in 32 bits
        y = _mlp(x[t].expand(k, -1).contiguous(), s["w_gate_up"][ids[t]], s["w_down"][ids[t]])
        out[t] = (weight[t][:, None] * y).sum(0)
    if s["ws_gate_up"] is not None:
        both = x @ s["ws_gate_up"].float().t()
        half = both.shape[1] // 2
        out = out + (_act(both[:, :half], "silu") * both[:, half:]) @ s["ws_down"].float().t()
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(torch.bfloat16)


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y if s["case"]["f32"] else y.to(torch.bfloat16)


def _plain_linear_bwd(s):
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _slope(s["z"].float(), s["case"]["act"])
    dx = (dz @ s["w"].float()).to(torch.bfloat16)
    dw = (dz.t() @ s["x"].float()).to(torch.bfloat16)
    return dx, dw, dz.sum(0) if s["bias"] is not None else None


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    far = x - mean[:, None]
    rstd = 1.0 / ((far * far).mean(1) + s["eps"]).sqrt()
    y = far * rstd[:, None] * s["w"].float() + s["b"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    dy, mean, rstd = s["dy"].float(), s["mean"][:, None], s["rstd"][:, None]
    xhat = (s["x"].float() - mean) * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0)


def run(s):
    kind = s["case"]["kind"]
    if own:
        if kind == "few":
            return s["layer"].forward(s["x"], logits=s["logits"], residual=s["residual"])
        if kind == "linear":
            return s["layer"].forward(s["x"], residual=s["residual"])
        if kind == "linear_bwd":
            return s["layer"].backward(s["dy"], s["x"], s["z"])
        if kind == "norm":
            return s["layer"].forward(s["x"], stats=True)
        return s["layer"].backward(s["dy"], s["x"], s["mean"], s["rstd"])
    return dict(few=_plain_few, linear=_plain_linear, linear_bwd=_plain_linear_bwd, norm=_plain_norm,
                norm_bwd=_plain_norm_bwd)[kind](s)


def work(case):
    kind = case["kind"]
    if kind == "few":
        T, E, k, H, F, Fs = (case[n] for n in ("T", "E", "k", "H", "F", "Fs"))
        touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that T tokens reach, on average
        weights = 2.0 * 3 * H * (touched * F + Fs)
        rows = 2.0 * T * H * (3 if case["residual"] else 2)
        return dict(bytes=weights + rows + 4.0 * T * E, flops=6.0 * T * H * (k * F + Fs))
    if kind in ("linear", "linear_bwd"):
        M, N, K = (float(case[n]) for n in "MNK")
        out = 4 if case["f32"] else 2
        if kind == "linear":
            moved = 2 * M * K + 2 * N * K + M * N * (out + (2 if case["res"] else 0)) + (4 * N if case["bias"] else 0)
            return dict(bytes=moved, flops=2 * M * N * K)
        moved = 4 * M * K + 4 * N * K + M * N * (out + (2 if case["act"] != "none" else 0)) + (4 * N if case["bias"] else 0)
        return dict(bytes=moved, flops=4 * M * N * K)
    M, H, size = float(case["M"]), float(case["H"]), 4 if case["f32"] else 2
    if kind == "norm":
        return dict(bytes=2 * M * H * size + 8 * M + 2 * H * size, flops=8 * M * H)
    return dict(bytes=3 * M * H * size + 8 * M + H * size + 8 * H, flops=14 * M * H)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    d = {n: v.double() for n, v in s.items() if torch.is_tensor(v) and not n.startswith("w_") and not n.startswith("ws_")}
    act = case.get("act", "none")
    if kind == "few":
        T, k, F, Fs = case["T"], case["k"], case["F"], case["Fs"]
        order = sorted(((-v, e, t) for t, row in enumerate(s["logits"].tolist()) for e, v in enumerate(row)),
                       key=lambda q: (q[2], q[0], q[1]))
        E = case["E"]
        mine = [order[t * E:t * E + k] for t in range(T)]
        out = torch.zeros_like(d["x"])
        by_expert = {}
        for t in range(T):
            top = torch.tensor([-q[0] for q in mine[t]], dtype=torch.float64)
            p = torch.softmax(top, 0) if case["score"] == "softmax" else torch.sigmoid(top) / torch.sigmoid(top).sum()
            for q, w in zip(mine[t], p.tolist()):
                by_expert.setdefault(q[1], []).append((t, w * s["scale"]))
        for e, rows in by_expert.items():
            at = torch.tensor([t for t, _ in rows], device="cuda")
            w = torch.tensor([v for _, v in rows], dtype=torch.float64, device="cuda")
            both = d["x"][at] @ s["w_gate_up"][e].double().t()
            h = torch.nn.functional.silu(both[:, :F]) * both[:, F:]
            out.index_add_(0, at, (h @ s["w_down"][e].double().t()) * w[:, None])
        if Fs:
            both = d["x"] @ s["ws_gate_up"].double().t()
            out += (torch.nn.functional.silu(both[:, :Fs]) * both[:, Fs:]) @ s["ws_down"].double().t()
        return out + d["residual"] if case["residual"] else out
    forms = dict(none=lambda v: v, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu)
    if kind == "linear":
        y = forms[act](torch.nn.functional.linear(d["x"], d["w"], d.get("bias")))
        return y + d["residual"] if case["res"] else y
    if kind == "linear_bwd":
        dz = d["dy"]
        if act != "none":
            z = d["z"].requires_grad_(True)
            dz = torch.autograd.grad(forms[act](z), z, dz)[0]
        return dz @ d["w"], dz.t() @ d["x"], dz.sum(0) if case["bias"] else None
    H, x = case["H"], d["x"]
    if kind == "norm":
        var, mean = torch.var_mean(x, 1, unbiased=False)
        return torch.nn.functional.layer_norm(x, (H,), d["w"], d["b"], s["eps"]), mean, torch.rsqrt(var + s["eps"])
    xhat = (x - d["mean"][:, None]) * d["rstd"][:, None]
    g = d["dy"] * d["w"]
    pull = (g.sum(1) / H)[:, None] + xhat * ((g * xhat).sum(1) / H)[:, None]
    return d["rstd"][:, None] * (g - pull), (d["dy"] * xhat).sum(0), d["dy"].sum(0)
