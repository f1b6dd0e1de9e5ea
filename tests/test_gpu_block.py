"""Norm, router and experts together, as a feed-forward block runs them."""
import pytest
import torch

from moe_routed_expert_top_b200.layer import FeedForwardBlock, LayerNorm, Linear, RoutedExperts
from tests import ops_ref as R
from tests.gpu_util import DEV, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(E=24, k=4, H=512, F=256, Fs=128):
    g = torch.Generator(device=DEV).manual_seed(0)
    n = lambda *s, sd=1.0, mean=0.0, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=DEV).normal_(
        mean, sd, generator=g)
    norm = LayerNorm(n(H, sd=0.1, mean=1.0), n(H, sd=0.1))
    router = Linear(n(E, H, sd=H ** -0.5), n(E, dt=torch.float32), out_dtype=torch.float32)
    routed = RoutedExperts(n(E, 2 * F, H, sd=0.04), n(E, H, F, sd=0.04), k, "sigmoid", True, 2.5,
                           ws_gate_up=n(2 * Fs, H, sd=0.04), ws_down=n(H, Fs, sd=0.04))
    return FeedForwardBlock(norm, router, routed), n


@pytest.mark.parametrize("T", [1, 3, 16, 64, 65, 200])
def test_block(T):
    block, n = make()
    x = n(T, 512, sd=2.0)
    out = block.forward(x)
    # step by step against 64 bits: each step on what the step before gave
    hidden = block.norm.forward(x)
    (ref, tol), _, _ = R.norm(x, block.norm.weight, block.norm.bias, block.norm.eps)
    R.check(hidden, ref, tol, "norm")
    logits = block.router.forward(hidden)
    ref, tol, _, _ = R.linear(hidden, block.router.weight, block.router.bias, "none", None, torch.float32)
    R.check(logits, ref, tol, "router")
    e = block.routed
    ids, w = e.route(logits)
    ref, tol = R.layer(hidden, ids, w, e.w_gate_up, e.w_down, e.scale, e.ws_gate_up, e.ws_down, x)
    if T > 64:  # the routed output is rounded before the residual is added
        tol = tol + R.half(torch.bfloat16) * (ref.abs() + x.double().abs() + tol)
        tol = tol + 1e-2 * (1 + ref.abs())  # the large forward's own tolerance
    R.check(out, ref, tol, "block")


def test_block_in_a_graph():
    block, n = make()
    x, y = n(8, 512), n(8, 512)
    want = block.forward(y)
    buf = x.clone()
    block.forward(buf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block.forward(buf)
    buf.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_block_of_no_tokens():
    block, n = make()
    assert block.forward(n(0, 512)).shape == (0, 512)


def test_block_graphs_of_two_sizes():
    """A graph keeps its workspace while larger calls, captured or not, come and go."""
    block, n = make()
    xs = {T: n(T, 512) for T in (80, 300)}
    want = {T: block.forward(x) for T, x in xs.items()}
    graphs, outs = {}, {}
    for T in (80, 300):
        block.forward(xs[T])
        torch.cuda.synchronize()
        graphs[T] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[T]):
            outs[T] = block.forward(xs[T])
    big = block.forward(n(900, 512))
    kept = [torch.full((1 << 20,), 7, dtype=torch.int32, device=DEV) for _ in range(16)]
    before = big.clone()
    for T in (80, 300, 80):
        graphs[T].replay()
    torch.cuda.synchronize()
    for T in (80, 300):
        assert torch.equal(outs[T], want[T])
    assert torch.equal(big, before) and all(bool((k == 7).all()) for k in kept)


def test_block_on_two_streams():
    block, n = make()
    xs = [n(200, 512) for _ in range(2)]
    want = [block.forward(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(block.forward(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_block_checks():
    block, n = make()
    with pytest.raises(ValueError):
        FeedForwardBlock(block.norm, Linear(n(24, 512)), block.routed)       # bf16 logits
    with pytest.raises(ValueError):
        FeedForwardBlock(LayerNorm(n(64)), block.router, block.routed)
