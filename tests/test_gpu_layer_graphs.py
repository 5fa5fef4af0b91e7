"""Layer steps in captured graphs where the node before a step is not one
kernel of the same stream: copies and fills, a fork of two streams and their
join, a step that follows two others.  The steps start before their
predecessor ends (csrc/launch.cuh); results must be an eager run's, to the bit.
"""
import pytest
import torch

from context_merge_gb300 import cpdr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    return cpdr.Context(1, 640, 1, 64, 1, dtype="bf16")


def tensors(seed, C=256):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=gen, device="cuda")

    return dict(x=randn(640, C).bfloat16(), norm=1 + 0.1 * randn(C), w=(randn(C, C) / 16).bfloat16(),
                v=(randn(C, C) / 16).bfloat16(), g=-randn(640, C).abs(), h0=randn(1, C))


def step(ctx, d, src, fork):
    """A copy, a norm, two products (on two streams with ``fork``) and a recurrence
    over the sum of both, a fill in between; every buffer is overwritten."""
    b = d["buf"]
    b["x"].copy_(src)                                        # a copy node
    ctx.rmsnorm_fwd(b["x"], d["norm"], y=b["n"])
    main = torch.cuda.current_stream()
    if fork:
        d["side"].wait_stream(main)
    with torch.cuda.stream(d["side"] if fork else main):
        ctx.linear_fwd(b["n"], d["v"], b["q"], activation="silu")
    ctx.linear_fwd(b["n"], d["w"], b["p"])
    if fork:
        main.wait_stream(d["side"])
    ctx.linear_fwd(b["p"], d["v"], b["r"], residual=b["q"])  # follows both
    b["y"].zero_()                                           # a fill node
    ctx.glr_fwd(b["r"][None], d["g"][None], b["y"][None], h0=d["h0"], hT=b["hT"])
    b["last"].copy_(b["y"])                                  # a copy behind a step
    return b["last"], b["hT"]


def prepared(seed, C=256):
    d = tensors(seed, C)
    d["buf"] = {k: torch.zeros_like(d["x"]) for k in ("x", "n", "p", "q", "r", "y", "last")}
    d["buf"]["hT"] = torch.zeros_like(d["h0"])
    d["side"] = torch.cuda.Stream()
    return d


@pytest.mark.parametrize("fork", [False, True])
def test_replays_equal_eager_runs(ctx, fork):
    d = prepared(1)
    sources = [tensors(s)["x"] for s in (5, 6, 7)]
    want = [[t.clone() for t in step(ctx, d, s, False)] for s in sources]
    torch.cuda.synchronize()
    src = torch.zeros_like(sources[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ctx, d, src, fork)
    for _ in range(3):
        for s, w in zip(sources, want):
            src.copy_(s)
            graph.replay()
            for a, b in zip(out, w):
                assert torch.equal(a, b)
    ctx.check_device_status()


def test_two_graphs_in_turn_and_eager_runs_between(ctx):
    a, b = prepared(2), prepared(3)
    src = tensors(8)["x"]
    want = [[t.clone() for t in step(ctx, d, src, False)] for d in (a, b)]
    graphs = []
    for d in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(ctx, d, src, True)
        graphs.append((g, out))
    for _ in range(5):
        for (g, out), d, w in zip(graphs, (a, b), want):
            g.replay()
            assert all(torch.equal(x, y) for x, y in zip(out, w))
            assert all(torch.equal(x, y) for x, y in zip(step(ctx, d, src, True), w))
    ctx.check_device_status()


def test_forked_streams_without_a_graph(ctx):
    d = prepared(4)
    src = tensors(9)["x"]
    want = [t.clone() for t in step(ctx, d, src, False)]
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(step(ctx, d, src, True), want))
