"""The few-token layer (moe_experts_forward_few): every element against a 64-bit
form over ragged sizes, skewed and repeated routings; its routing bit for bit
against moe_route_topk; streams, graphs, aliasing and offsets past 32 bits."""
import pytest
import torch

import moe_routed_expert_top_b200 as M
from moe_routed_expert_top_b200.layer import FewTokenExperts
from tests import ops_ref as R
from tests.gpu_util import DEV, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(T, E, k, H, F, Fs=0, seed=0, std=0.05):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s, sd=1.0, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=DEV).normal_(0, sd, generator=g)
    return dict(x=n(T, H), logits=n(T, E, dt=torch.float32), wgu=n(E, 2 * F, H, sd=std), wd=n(E, H, F, sd=std),
                sgu=n(2 * Fs, H, sd=std) if Fs else None, sd=n(H, Fs, sd=std) if Fs else None, res=n(T, H))


def route(s, k, score="softmax", renorm=True):
    T, E = s["logits"].shape
    p = M.make_problem(T=T, H=64, F=64, E=E, top_k=k, score_fn=score, renormalize=renorm)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, dtype=torch.float32, device=DEV)
    M.moe_route_topk(p, s["logits"], ids, w)
    return ids, w


def expected(s, ids, w, scale=1.0, residual=True):
    return R.layer(s["x"], ids, w, s["wgu"], s["wd"], scale, s["sgu"], s["sd"], s["res"] if residual else None)


@pytest.mark.parametrize("T,E,k,H,F,Fs,score,renorm", [
    (1, 1, 1, 64, 64, 0, "softmax", True),
    (1, 8, 2, 128, 64, 64, "sigmoid", True),
    (2, 5, 5, 192, 320, 0, "softmax", False),
    (7, 33, 3, 2368, 128, 0, "softmax", True),      # 16 output rows a CTA
    (8, 6, 2, 2432, 192, 128, "sigmoid", False),    # 17
    (9, 16, 4, 576, 768, 0, "softmax", True),
    (16, 4, 2, 320, 448, 64, "softmax", True),
    (17, 4, 1, 1024, 128, 256, "sigmoid", True),    # the shared expert in two token groups
    (33, 7, 7, 64, 192, 0, "softmax", True),        # every token at every expert: 33 rows each
    (64, 3, 2, 512, 64, 64, "sigmoid", True),
    (64, 257, 9, 128, 128, 0, "softmax", False),
    (64, 1024, 32, 64, 64, 0, "sigmoid", True),
    (3, 1024, 32, 64, 128, 64, "softmax", True),
    (5, 12, 3, 5056, 704, 0, "softmax", True),      # 35 rows a CTA: two passes
])
def test_layer_from_logits(T, E, k, H, F, Fs, score, renorm):
    s = make(T, E, k, H, F, Fs, seed=T + E)
    L = FewTokenExperts(s["wgu"], s["wd"], k, score, renorm, 1.5, s["sgu"], s["sd"])
    ids = torch.full((T, k), -9, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -9.0, dtype=torch.float32, device=DEV)
    out = L.forward(s["x"], ids, w, logits=s["logits"], residual=s["res"])
    rids, rw = route(s, k, score, renorm)
    assert torch.equal(ids, rids)
    assert torch.equal(w.view(torch.int32), rw.view(torch.int32))
    R.check(out, *expected(s, rids, rw, 1.5), "layer")
    assert L.device_status() == 0
    # given the ids and weights instead: the same bits
    again = L.forward(s["x"], rids, rw, residual=s["res"])
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_ties_and_minus_infinity():
    T, E, k = 12, 40, 8
    s = make(T, E, k, 128, 64)
    s["logits"] = (s["logits"] * 2).round() / 2           # many ties
    s["logits"][3] = 0.0
    s["logits"][4, 10:] = -torch.inf
    s["logits"][5, 5] = -0.0
    L = FewTokenExperts(s["wgu"], s["wd"], k)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, dtype=torch.float32, device=DEV)
    out = L.forward(s["x"], ids, w, logits=s["logits"])
    rids, rw = route(s, k)
    assert torch.equal(ids, rids) and torch.equal(w.view(torch.int32), rw.view(torch.int32))
    R.check(out, *expected(s, rids, rw, residual=False))


def test_nan_logits_stay_inside():
    s = make(4, 40, 4, 64, 64)
    s["logits"][1] = torch.nan
    s["logits"][2] = -torch.nan
    s["logits"].view(torch.int32)[3] = -1                  # the NaN of all ones
    L = FewTokenExperts(s["wgu"], s["wd"], 4)
    ids = torch.full((4, 4), -9, dtype=torch.int32, device=DEV)
    w = torch.empty(4, 4, dtype=torch.float32, device=DEV)
    out = L.forward(s["x"], ids, w, logits=s["logits"])
    torch.cuda.synchronize()
    assert int(ids.min()) >= 0 and int(ids.max()) < 40
    assert torch.isfinite(out[0]).all()


@pytest.mark.parametrize("kind", ["one expert", "repeated", "bad", "none"])
def test_given_routings(kind):
    T, E, k, H, F = 41, 6, 4, 256, 192
    s = make(T, E, k, H, F, 64, seed=5)
    g = torch.Generator(device=DEV).manual_seed(9)
    ids = torch.randint(0, E, (T, k), device=DEV, generator=g, dtype=torch.int32)  # repeats happen
    if kind == "one expert":
        ids = torch.full_like(ids, E - 1)
    elif kind == "bad":
        ids[::3, 1] = E
        ids[1::5, 0] = -1
        ids[2, 2] = 2 ** 31 - 1
        ids[7, 3] = -2 ** 31
        ids[9] = E + 7                                     # a token with no expert at all
    elif kind == "none":
        ids = torch.full_like(ids, -1)
    w = torch.rand(T, k, device=DEV, generator=g)
    L = FewTokenExperts(s["wgu"], s["wd"], k, routed_scaling_factor=2.5, ws_gate_up=s["sgu"], ws_down=s["sd"])
    out = L.forward(s["x"], ids, w, residual=s["res"])
    R.check(out, *expected(s, ids, w, 2.5), kind)
    flag = M.MOE_DEV_BAD_EXPERT_ID if kind in ("bad", "none") else 0
    assert L.device_status() == flag


def test_no_expert_without_shared_or_residual_is_zero():
    s = make(3, 4, 2, 128, 64)
    ids = torch.full((3, 2), 99, dtype=torch.int32, device=DEV)
    L = FewTokenExperts(s["wgu"], s["wd"], 2)
    out = L.forward(s["x"], ids, torch.ones(3, 2, device=DEV), out=torch.full_like(s["x"], torch.nan))
    assert (out == 0).all()


def test_infinite_weight_of_another_expert_is_not_touched():
    s = make(2, 3, 1, 128, 64)
    s["wd"][2] = torch.inf
    s["wgu"][2] = torch.nan
    ids = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    out = FewTokenExperts(s["wgu"], s["wd"], 1).forward(s["x"], ids, torch.ones(2, 1, device=DEV))
    assert torch.isfinite(out).all()
    ids[1, 0] = 2  # token 1 meets it, token 0 does not
    out = FewTokenExperts(s["wgu"], s["wd"], 1).forward(s["x"], ids, torch.ones(2, 1, device=DEV))
    assert torch.isfinite(out[0]).all() and not torch.isfinite(out[1]).any()


@pytest.mark.parametrize("T", [1, 64])
def test_out_may_be_hidden_or_residual(T):
    s = make(T, 8, 2, 320, 128, 64, seed=T)
    L = FewTokenExperts(s["wgu"], s["wd"], 2, ws_gate_up=s["sgu"], ws_down=s["sd"])
    want = L.forward(s["x"], logits=s["logits"], residual=s["res"])
    r = s["res"].clone()
    assert torch.equal(L.forward(s["x"], logits=s["logits"], residual=r, out=r), want)
    want = L.forward(s["x"], logits=s["logits"], residual=s["x"])
    x = s["x"].clone()
    assert torch.equal(L.forward(x, logits=s["logits"], residual=x, out=x), want)


def test_rows_behind_the_last_token_stay():
    s = make(5, 8, 2, 192, 64)
    whole = torch.full((9, 192), 7.0, dtype=torch.bfloat16, device=DEV)
    FewTokenExperts(s["wgu"], s["wd"], 2).forward(s["x"], logits=s["logits"], out=whole[:5])
    assert (whole[5:] == 7.0).all()


def test_streams_and_repeats_give_the_same_bits():
    s = make(13, 16, 4, 768, 256, 128)
    L = FewTokenExperts(s["wgu"], s["wd"], 4, ws_gate_up=s["sgu"], ws_down=s["sd"])
    want = L.forward(s["x"], logits=s["logits"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(L.forward(s["x"], logits=s["logits"]))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


def test_graphs_replay_on_new_inputs():
    s, t = make(6, 16, 4, 512, 256, 64), make(6, 16, 4, 512, 256, 64, seed=1)
    L = FewTokenExperts(s["wgu"], s["wd"], 4, ws_gate_up=s["sgu"], ws_down=s["sd"])
    x, lg = s["x"].clone(), s["logits"].clone()
    L.forward(x, logits=lg)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of one layer object
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a = L.forward(x, logits=lg)
            b = L.forward(a, logits=lg, residual=x)
        graphs.append((g, b))
    for src in (t, s):
        x.copy_(src["x"])
        lg.copy_(src["logits"])
        want = L.forward(L.forward(x, logits=lg), logits=lg, residual=x)
        for g, b in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, b in graphs:
            assert torch.equal(b.view(torch.int16), want.view(torch.int16))


def test_weights_past_32_bit_offsets():
    E, F, H = 40, 4096, 8192                               # 2.7e9 values of w_gate_up
    g = torch.Generator(device=DEV).manual_seed(3)
    wgu = torch.empty(E, 2 * F, H, dtype=torch.bfloat16, device=DEV).normal_(0, 0.02, generator=g)
    wd = torch.empty(E, H, F, dtype=torch.bfloat16, device=DEV).normal_(0, 0.02, generator=g)
    x = torch.empty(3, H, dtype=torch.bfloat16, device=DEV).normal_(0, 1, generator=g)
    ids = torch.tensor([[E - 1, 0], [E - 2, E - 1], [33, 39]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, 0.5], [0.25, 0.75], [1.0, 0.0]], device=DEV)
    out = FewTokenExperts(wgu, wd, 2).forward(x, ids, w)
    R.check(out, *R.layer(x, ids, w, wgu, wd, 1.0))


def test_agrees_with_the_large_forward():
    from moe_routed_expert_top_b200.layer import RoutedExperts
    s = make(64, 32, 4, 1024, 512, 256, seed=2, std=0.02)
    ids, w = route(s, 4, "sigmoid")
    big = RoutedExperts(s["wgu"], s["wd"], 4, "sigmoid", True, 2.5, ws_gate_up=s["sgu"], ws_down=s["sd"])
    few = FewTokenExperts(s["wgu"], s["wd"], 4, "sigmoid", True, 2.5, s["sgu"], s["sd"])
    ref, tol = expected(s, ids, w, 2.5, residual=False)
    a, b = big.forward(s["x"], ids, w), few.forward(s["x"], ids, w)
    R.check(b, ref, tol)
    assert ((a.double() - b.double()).abs() <= 2 * tol).all()
