"""The layer steps run together, as a layer around a token mixer uses them:
residual and norm, products, causal conv, gated linear recurrence or delta
rule, output product onto the residual stream -- a forward and its gradients
in training form, and decoding token by token in serving form.

The gradients of the whole chain are compared with differences of the chain
itself in 64 bits (the oracle's functions composed), decoding with the
prefill of the same tokens.
"""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import conv as oconv
from oracle import layer_steps as ol

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def weights(D, C, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=gen)

    return dict(norm=1 + 0.2 * randn(D), w_in=(randn(C, D) / D ** 0.5).bfloat16(), b_in=0.1 * randn(C),
                w_gate=(randn(C, D) / D ** 0.5).bfloat16(), b_gate=4 + 0.5 * randn(C),
                conv=randn(C, 4) / 2, w_out=(randn(D, C) / C ** 0.5).bfloat16())


def cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def test_training_chain_gradients():
    """norm -> product with SiLU -> recurrence -> output product + residual over a packed batch."""
    D, C, lengths = 64, 136, [37, 0, 150, 13]
    cu = np.cumsum([0] + lengths).tolist()
    T = cu[-1]
    w = weights(D, C)
    gen = torch.Generator().manual_seed(1)
    x, delta, dy = (torch.randn((1, T, D), generator=gen).bfloat16() for _ in range(3))
    g = torch.nn.functional.logsigmoid(2 + torch.randn((1, T, C), generator=gen))
    ctx = cpdr.Context(1, T, 1, 64, 1, dtype="bf16", cu_seqlens=cu)
    c, xd, dd, dyd, gd = cuda(w), x.cuda(), delta.cuda(), dy.cuda(), g.cuda()
    bf = dict(device="cuda", dtype=torch.bfloat16)
    s, n = torch.empty_like(xd), torch.empty_like(xd)
    ctx.rmsnorm_fwd(xd, c["norm"], residual=dd, sum_out=s, y=n, eps=EPS)
    u, z, h = (torch.empty(1, T, C, **bf) for _ in range(3))
    ctx.linear_fwd(n, c["w_in"], u, bias=c["b_in"], activation="silu", z=z)
    carry = torch.empty(ctx.glr_carry_shape(C), device="cuda")
    ctx.glr_fwd(u, gd, h, carry=carry)
    y = torch.empty_like(xd)
    ctx.linear_fwd(h, c["w_out"], y, residual=s)
    # backward: dy reaches the output product and, past it, the residual stream s
    o = ctx.linear_bwd(h, c["w_out"], dyd, out=dict(dx=torch.empty_like(h), dw=torch.empty_like(c["w_out"])))
    r = ctx.glr_bwd(u, gd, carry, o["dx"])
    i = ctx.linear_bwd(n, c["w_in"], r["dx"], z=z, activation="silu")
    b = ctx.rmsnorm_bwd(s, c["norm"], i["dx"], dsum=dyd, eps=EPS)
    torch.cuda.synchronize()
    ctx.check_device_status()

    # the same chain in 64 bits, rounded where the kernels round
    def q(a):
        return torch.from_numpy(np.ascontiguousarray(a)).bfloat16().double().numpy()

    s64 = q(ol.as64(x)[0] + ol.as64(delta)[0])
    n64 = q(ol.rmsnorm_forward(ol.as64(x)[0], w["norm"], EPS, ol.as64(delta)[0])["y"])
    f = ol.linear_forward(n64, w["w_in"], w["b_in"], "silu")
    u64, z64 = q(f["y"]), q(f["z"])
    h64 = q(ol.glr_forward(u64[None], g, cu_seqlens=cu)["y"][0])
    y64 = ol.linear_forward(h64, w["w_out"], residual=s64)["y"]
    go = ol.linear_backward(h64, w["w_out"], dy[0])
    gr = ol.glr_backward(u64[None], g, q(go["dx"])[None], cu_seqlens=cu)
    gi = ol.linear_backward(n64, w["w_in"], q(gr["dx"][0]), z64, "silu")
    gb = ol.rmsnorm_backward(s64, w["norm"], EPS, q(gi["dx"]), dy[0])
    # roundings of bf16 tensors along the chain, each 2^-8 of a value at most and
    # independent of one another: under eight of them at any output
    for got, ref in ((y[0], y64), (o["dw"], go["dw"]), (r["dg"][0], gr["dg"][0]), (i["dw"], gi["dw"]),
                     (i["dbias"], gi["dbias"]), (b["ds"][0], gb["ds"]), (b["dweight"], gb["dweight"])):
        got = got.double().cpu().numpy()
        assert np.linalg.norm(got - ref) <= 8 * 2.0 ** -8 * np.linalg.norm(ref)


def test_prefill_in_8_bits_then_decode_equals_prefill():
    """norm with e4m3 output -> e4m3 products (input and gate) -> recurrence -> output product; the first
    tokens of every sequence as a prefill, the rest token by token over a shuffled pool of slots with an
    empty row in the batch, against one prefill of all tokens."""
    B, T, P, D, C = 5, 12, 7, 64, 72
    w = weights(D, C, 3)
    c = cuda(w)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((B, T, D), generator=gen).bfloat16().cuda()

    def to8(t):
        s = (t.float().abs().amax(1) / 448.0)
        return (t.float() / s[:, None]).to(torch.float8_e4m3fn), s

    win, sin = to8(c["w_in"])
    wg, sg = to8(c["w_gate"])

    def mixer_inputs(ctx, xs):
        n8 = torch.empty(xs.shape, dtype=torch.float8_e4m3fn, device="cuda")
        ns = torch.empty(xs.shape[:-1], device="cuda")
        ctx.rmsnorm_fwd(xs, c["norm"], y8=n8, scale=ns, eps=EPS)
        u, gate = (torch.empty(*xs.shape[:-1], C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ctx.linear_fwd(n8, win, u, bias=c["b_in"], activation="gelu", x_scale=ns, w_scale=sin)
        ctx.linear_fwd(n8, wg, gate, bias=c["b_gate"], x_scale=ns, w_scale=sg)
        return u, torch.nn.functional.logsigmoid(gate.float())

    def prefill(tokens, state):
        ctx = cpdr.Context(B, tokens, 1, 64, 1, dtype="bf16")
        xs = x[:, :tokens].contiguous()
        u, g = mixer_inputs(ctx, xs)
        h, y = torch.empty_like(u), torch.empty_like(xs)
        ctx.glr_fwd(u, g, h, h0=state, hT=state)
        ctx.linear_fwd(h, c["w_out"], y, residual=xs)
        return y

    whole = torch.zeros(B, C, device="cuda")
    ref = prefill(T, whole)
    part = torch.zeros(B, C, device="cuda")
    first = prefill(P, part)
    slots = torch.tensor([6, 2, 7, 0, 5], dtype=torch.int32, device="cuda")
    pool = torch.full((8, C), 99.0, device="cuda")
    pool[slots.long()] = part
    rows = torch.cat([slots[:2], torch.tensor([-1], dtype=torch.int32, device="cuda"), slots[2:]])
    live = torch.tensor([0, 1, 3, 4, 5], device="cuda")
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    outs = []
    for t in range(P, T):
        xs = torch.zeros(B + 1, D, dtype=torch.bfloat16, device="cuda")
        xs[live] = x[:, t]
        u, g = mixer_inputs(ctx, xs)
        h, y = torch.zeros_like(u), torch.empty_like(xs)
        ctx.glr_step(u, g, pool, h, slots=rows)
        ctx.linear_fwd(h, c["w_out"], y, residual=xs)
        outs.append(y[live])
    torch.cuda.synchronize()
    ctx.check_device_status()
    assert torch.equal(first, ref[:, :P])               # the same rows, the same bits
    assert (pool[[1, 3, 4]] == 99).all()                # slots of no row
    dec = torch.stack(outs, 1)
    # the products of few rows add in another order (2^-24 of the sums), which
    # can move a rounding to bf16 by a whole step, 2 x 2^-8 of a value
    assert (dec.double() - ref[:, P:].double()).norm() <= 2.0 ** -8 * ref[:, P:].double().norm()
    assert (pool[slots.long()].double() - whole.double()).norm() <= 2.0 ** -8 * whole.double().norm()


def test_norm_product_and_conv_feed_the_delta_rule():
    """The q, k, v inputs of a delta-rule layer by the layer steps: norm -> product -> conv on the context's
    segments -> delta rule; heads normalised; output product onto the residual."""
    T, H, d, D, R = 512, 2, 128, 128, 4
    gen = torch.Generator().manual_seed(6)

    def randn(*s):
        return torch.randn(s, generator=gen)

    x = randn(1, T, D).bfloat16()
    wqkv, wo = (randn(3 * H * d, D) / D ** 0.5).bfloat16(), (randn(D, H * d) / (H * d) ** 0.5).bfloat16()
    cw, ones, hn = randn(3 * H * d, 4) / 2, torch.ones(D), 1 + 0.1 * randn(d)
    beta = torch.sigmoid(randn(1, T, H)).bfloat16()
    g = torch.nn.functional.logsigmoid(3 + randn(1, T, H))
    ctx = cpdr.Context(1, T, H, d, R, dtype="bf16", conv_width=4)
    xd = x.cuda()
    n, qkv = torch.empty_like(xd), torch.empty(1, T, 3 * H * d, dtype=torch.bfloat16, device="cuda")
    ctx.rmsnorm_fwd(xd, ones.cuda(), y=n, eps=EPS)
    ctx.linear_fwd(n, wqkv.cuda(), qkv)
    y = torch.empty_like(qkv)
    ctx.conv1d_fwd(qkv, cw.cuda(), None, y)
    q, k, v = (t.reshape(1, T, H, d).contiguous() for t in y.split(H * d, dim=2))
    unit = torch.full((d,), d ** -0.5, device="cuda")
    ctx.rmsnorm_fwd(q, unit, y=q, eps=EPS)              # in place: unit vectors per head
    ctx.rmsnorm_fwd(k, unit, y=k, eps=EPS)
    o, _ = ctx.run(q, k, v, beta.cuda(), g.cuda())
    ctx.rmsnorm_fwd(o, hn.cuda(), y=o, eps=EPS)
    out = torch.empty_like(xd)
    ctx.linear_fwd(o.view(1, T, H * d), wo.cuda(), out, residual=xd)
    torch.cuda.synchronize()
    ctx.check_device_status()

    def r(a):
        return torch.from_numpy(np.ascontiguousarray(a)).bfloat16().double().numpy()

    import oracle
    n64 = r(ol.rmsnorm_forward(x[0], ones, EPS)["y"])
    y64 = r(oconv.causal_conv1d(r(ol.linear_forward(n64, wqkv)["y"])[None], cw, None))[0]
    parts = [p.reshape(T * H, d) for p in np.split(y64, 3, axis=1)]
    q64, k64 = (r(ol.rmsnorm_forward(p, np.full(d, d ** -0.5), EPS)["y"]).reshape(1, T, H, d) for p in parts[:2])
    def b16(a):
        return torch.from_numpy(np.ascontiguousarray(a)).bfloat16()

    o64 = oracle.Problem(b16(q64), b16(k64), b16(parts[2].reshape(1, T, H, d)), beta, g).segmented(R)["o"]
    h64 = r(ol.rmsnorm_forward(r(o64).reshape(T * H, d), hn, EPS)["y"]).reshape(T, H * d)
    ref = ol.linear_forward(h64, wo, residual=x[0])["y"]
    # the delta rule's own bar (2e-2), and the roundings of six bf16 tensors around it
    err = np.linalg.norm(out[0].double().cpu().numpy() - ref) / np.linalg.norm(ref)
    assert err <= 2e-2 + 6 * 2.0 ** -8, err


def test_a_decoding_step_as_one_graph():
    """norm -> product -> step -> output product captured once and replayed over changing inputs."""
    n, D, C, S = 6, 128, 264, 16
    w = weights(D, C, 8)
    c = cuda(w)
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(n, D, generator=gen, device="cuda").bfloat16()
    gate = -torch.rand(n, C, generator=gen, device="cuda")
    slots = torch.tensor([3, 9, -1, 0, 15, 7], dtype=torch.int32, device="cuda")
    state = torch.randn(S, C, generator=gen, device="cuda")
    nrm, u, h, y = (torch.zeros(n, m, dtype=torch.bfloat16, device="cuda") for m in (D, C, C, D))

    def go():
        ctx.rmsnorm_fwd(x, c["norm"], y=nrm, eps=EPS)
        ctx.linear_fwd(nrm, c["w_in"], u, bias=c["b_in"], activation="silu")
        ctx.glr_step(u, gate, state, h, slots=slots)
        ctx.linear_fwd(h, c["w_out"], y, residual=x)

    begin = state.clone()
    go()                                                # sets the kernels up before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    xs = [torch.randn(n, D, generator=gen, device="cuda").bfloat16() for _ in range(4)]
    state.copy_(begin)
    want = []
    for t in xs:
        x.copy_(t)
        go()
        want.append((y.clone(), state.clone()))
    state.copy_(begin)
    for t, (wy, ws) in zip(xs, want):
        x.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(state, ws)
    ctx.check_device_status()


def test_two_graphs_that_share_a_workspace_run_one_after_the_other():
    """Two captured backwards over one workspace, replayed in turn on one stream."""
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    gen = torch.Generator(device="cuda").manual_seed(10)

    def rb(*s):
        return torch.randn(s, generator=gen, device="cuda").bfloat16()

    wt = rb(136, 64)
    ws = torch.empty(ctx.linear_bwd_workspace_bytes(200, 64, 136, "gelu"), dtype=torch.uint8, device="cuda")
    sets = [dict(x=rb(200, 64), dy=rb(200, 136), z=rb(200, 136)) for _ in range(2)]
    ref = [ctx.linear_bwd(s["x"], wt, s["dy"], z=s["z"], activation="gelu") for s in sets]
    graphs, outs = [], []
    for s in sets:
        out = {k: torch.zeros_like(v) for k, v in ref[0].items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ctx.linear_bwd(s["x"], wt, s["dy"], z=s["z"], activation="gelu", out=out, workspace=ws)
        graphs.append(graph)
        outs.append(out)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref, outs):
        for k in a:
            assert torch.equal(a[k], b[k]), k


def test_what_a_call_makes_belongs_to_the_stream_it_runs_on():
    """Backwards on a stream of their own, whose workspaces and outputs are made by the call, while the
    current stream keeps taking and filling memory."""
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    gen = torch.Generator(device="cuda").manual_seed(11)

    def rb(*s):
        return torch.randn(s, generator=gen, device="cuda").bfloat16()

    x, wt, dy, z = rb(3000, 264), rb(520, 264), rb(3000, 520), rb(3000, 520)
    w = torch.ones(520, device="cuda")
    lin = ctx.linear_bwd(x, wt, dy, z=z, activation="silu")
    norm = ctx.rmsnorm_bwd(z, w, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(8):
        got.append((ctx.linear_bwd(x, wt, dy, z=z, activation="silu", stream=side),
                    ctx.rmsnorm_bwd(z, w, dy, stream=side)))
        for _ in range(4):
            torch.full((3000 * 520 * 2 + 4096,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(a[k], lin[k]) for k in lin) and all(torch.equal(b[k], norm[k]) for k in norm)


def test_calls_on_two_streams_at_once():
    """The same context on two streams whose work overlaps: nothing is shared but the status word."""
    ctx = cpdr.Context(1, 2000, 1, 64, 1, dtype="bf16")
    gen = torch.Generator(device="cuda").manual_seed(12)
    sets = []
    for _ in range(2):
        x = torch.randn((1, 2000, 264), generator=gen, device="cuda").bfloat16()
        g = -torch.rand((1, 2000, 264), generator=gen, device="cuda")
        w = torch.randn((264, 264), generator=gen, device="cuda").bfloat16()
        sets.append((x, g, w))

    def go(x, g, w):
        u, h, few = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x[:, :7])
        ctx.linear_fwd(x, w, u, activation="gelu")
        ctx.glr_fwd(u, g, h)
        ctx.linear_fwd(x[:, :7].contiguous(), w, few)
        ctx.rmsnorm_fwd(h, torch.ones(264, device="cuda"), y=h)
        return u, h, few

    ref = [go(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(5):
        for i, (st, s) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(st):
                outs[i].append(go(*s))
    torch.cuda.synchronize()
    ctx.check_device_status()
    for r, many in zip(ref, outs):
        for one in many:
            assert all(torch.equal(a, b) for a, b in zip(r, one))


def test_a_chain_of_calls_equals_the_calls_one_by_one():
    """Kernels may begin while the one before them ends: a long chain of calls, each reading what the one
    before wrote (and writing what it read), against the same calls with a synchronisation after each."""
    D, C, S = 136, 264, 9
    w = cuda(weights(D, C, 21))
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    seq = cpdr.Context(1, 700, 1, 64, 1, dtype="bf16")

    def chain(wait):
        gen = torch.Generator(device="cuda").manual_seed(22)
        x = torch.randn((700, D), generator=gen, device="cuda").bfloat16()
        g = -torch.rand((1, 700, C), generator=gen, device="cuda")
        state, carry = torch.zeros(S, C, device="cuda"), torch.empty(seq.glr_carry_shape(C), device="cuda")
        n, few, u, h = x.clone(), x[:S].clone(), *(torch.zeros(700, C, device="cuda").bfloat16() for _ in range(2))
        ws = torch.empty(ctx.linear_bwd_workspace_bytes(700, D, C, "silu"), dtype=torch.uint8, device="cuda")
        grads = dict(dx=torch.empty_like(x), dw=torch.empty_like(w["w_in"]), dbias=torch.empty(C, device="cuda"))
        out = []

        def step(f, *a, **k):
            f(*a, **k)
            if wait:
                torch.cuda.synchronize()

        for _ in range(12):
            step(ctx.rmsnorm_fwd, x, w["norm"], y=n)
            step(ctx.linear_fwd, n, w["w_in"], u, bias=w["b_in"], activation="silu", z=h)
            step(ctx.linear_bwd, n, w["w_in"], u, z=h, activation="silu", out=grads, workspace=ws)
            step(seq.glr_fwd, u.view(1, 700, C), g, h.view(1, 700, C), carry=carry)
            step(ctx.linear_fwd, h, w["w_out"], x, residual=x)
            step(ctx.rmsnorm_fwd, few, w["norm"], residual=x[:S], sum_out=few, y=n[:S])
            step(ctx.linear_fwd, n[:S], w["w_in"], u[:S])
            step(ctx.glr_step, u[:S], g[0, :S], state, h[:S])
            step(ctx.linear_fwd, h[:S], w["w_out"], few, residual=few)
            out += [t.clone() for t in (x, few, state, carry, *grads.values())]
        torch.cuda.synchronize()
        return out

    for a, b in zip(chain(True), chain(False)):
        assert torch.equal(a, b)
