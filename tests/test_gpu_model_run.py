"""The model steps run together, as a delta-rule model uses them: tokens to
their embedding, layer norm, projections, causal conv and delta rule, and the
output onto the residual stream.  Decoding from pools of slots is compared with
the prefill of the same tokens, a training step's gradients with the chain in 64
bits; graphs, streams and shared workspaces with eager runs, to the bit.
"""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol
from oracle import model_steps as om

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


class Model:
    """Embedding -> [layer norm -> q, k, v -> causal conv -> delta rule -> output + residual]."""

    def __init__(self, V=300, D=128, H=2, d=128, W=4, G=2, gate="gdn", v_first=False, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def randn(*s):
            return torch.randn(s, generator=gen)

        self.D, self.H, self.d, self.W, self.G, self.gate, self.v_first = D, H, d, W, G, gate, v_first
        C = self.C = (G + 2) * H * d
        self.w = {k: v.cuda() for k, v in dict(
            table=randn(V, D).bfloat16(), norm=1 + 0.2 * randn(D), bias=0.1 * randn(D),
            qkv=(randn(C, D) / D ** 0.5).bfloat16(), conv=randn(C, W) / 2, conv_b=0.1 * randn(C),
            unit=torch.full((d,), d ** -0.5), out=(randn(D, G * H * d) / (G * H * d) ** 0.5).bfloat16()).items()}

    def context(self, B, T, R=1):
        return cpdr.Context(B, T, self.H, self.d, R, gate=self.gate, dtype="bf16", Hq=self.G * self.H,
                            state_v_first=self.v_first, conv_width=self.W)

    def new(self, *shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

    def inputs(self, ctx, tokens):
        """The residual stream and the conv's input of tokens [.., n]."""
        x, n, u = self.new(*tokens.shape, self.D), self.new(*tokens.shape, self.D), self.new(*tokens.shape, self.C)
        ctx.embed_fwd(tokens, self.w["table"], x, scale=0.5)
        ctx.layernorm_fwd(x, self.w["norm"], bias=self.w["bias"], y=n, eps=EPS)
        ctx.linear_fwd(n, self.w["qkv"], u)
        return x, u

    def heads(self, ctx, y):
        """q, k, v of the conv's output, q and k of unit length."""
        q, k, v = y.split([self.G * self.H * self.d, self.H * self.d, self.H * self.d], dim=-1)
        q = q.reshape(*y.shape[:-1], self.G * self.H, self.d).contiguous()
        k, v = (t.reshape(*y.shape[:-1], self.H, self.d).contiguous() for t in (k, v))
        ctx.rmsnorm_fwd(q, self.w["unit"], y=q)
        ctx.rmsnorm_fwd(k, self.w["unit"], y=k)
        return q, k, v

    def output(self, ctx, o, x):
        y = self.new(*x.shape)
        ctx.linear_fwd(o.reshape(*x.shape[:-1], -1), self.w["out"], y, residual=x)
        return y


def gates(m, n, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    beta = torch.sigmoid(torch.randn((*n, m.H), generator=gen, device="cuda")).bfloat16()
    g = torch.nn.functional.logsigmoid(3 + torch.randn((*n, m.H, *([m.d] if m.gate == "kda" else [])), generator=gen, device="cuda"))
    return beta, g


@pytest.mark.parametrize("gate,v_first", [("gdn", False), ("gdn", True), ("kda", False), ("kda", True)])
def test_prefill_then_decode_equals_prefill(gate, v_first):
    """The first tokens of every sequence as a prefill in chunk form, which leaves its states and the conv's
    windows; the rest from shuffled pools of slots, one token at a time and then three drafted ones at once,
    with an empty row in the batch; against one prefill of all tokens."""
    B, T, P, steps = 3, 75, 70, 2
    m = Model(gate=gate, v_first=v_first)
    tokens = torch.randint(0, 300, (B, T), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    beta, g = gates(m, (B, T))

    def prefill(n):
        ctx = m.context(B, n)
        x, u = m.inputs(ctx, tokens[:, :n].contiguous())
        y = torch.empty_like(u)
        ctx.conv1d_fwd(u, m.w["conv"], m.w["conv_b"], y)
        q, k, v = m.heads(ctx, y)
        o, bufs = ctx.run(q, k, v, beta[:, :n].contiguous(), g[:, :n].contiguous())
        return m.output(ctx, o, x), bufs["final_state"], u

    ref, ref_state, _ = prefill(T)
    _, state, u = prefill(P)
    slots = [4, 0, 6]
    pool = torch.full((8, *state.shape[1:]), 99.0, device="cuda")
    windows = torch.full((8, m.W - 1, m.C), 7.0, device="cuda").bfloat16()
    pool[slots], windows[slots] = state, u[:, P - (m.W - 1):]
    ctx = m.context(1, 1)

    def decode(rows, toks, b, gg):
        """rows: slot of each row; the tokens' outputs."""
        sl = torch.tensor(rows, dtype=torch.int32, device="cuda")
        x, u = m.inputs(ctx, toks)
        y = torch.zeros_like(u)
        ctx.conv1d_step(u, m.w["conv"], m.w["conv_b"], windows, y, slots=sl)
        q, k, v = m.heads(ctx, y)
        o = torch.zeros_like(q)
        ctx.delta_step(q, k, v, b, gg, pool, o, slots=sl)
        return m.output(ctx, o, x)

    outs = []
    for t in range(P, P + steps):
        at = [0, 1, 1, 2]     # row 1 is empty: the padding token, no slot
        toks = tokens[at, t].clone()
        toks[1] = -1
        outs.append(decode([slots[0], -1, slots[1], slots[2]], toks, beta[at, t].contiguous(), g[at, t].contiguous())[[0, 2, 3]])
    left = list(range(P + steps, T))
    seq = [0, 1, 2] * len(left)                                    # the sequences' tokens in turn
    pos = [t for t in left for _ in range(B)]
    drafted = decode([slots[s] for s in seq], tokens[seq, pos], beta[seq, pos].contiguous(), g[seq, pos].contiguous())
    outs += [drafted[i * B:(i + 1) * B] for i in range(len(left))]
    torch.cuda.synchronize()
    ctx.check_device_status()
    got = torch.stack(outs, 1).double()
    assert (pool[[1, 2, 3, 5, 7]] == 99).all() and (windows[[1, 2, 3, 5, 7]] == 7).all()
    # the chunk form takes its products in bf16 (its own bar against 64 bits is 2e-2 of the states and outputs)
    assert (got - ref[:, P:].double()).norm() <= 2e-2 * ref[:, P:].double().norm()
    assert (pool[slots].double() - ref_state.double()).norm() <= 2e-2 * ref_state.double().norm()


def test_drafted_tokens_at_once_equal_them_one_by_one():
    """Rows of one slot in one call, or in calls of their own: the same bits."""
    for gate, v_first in (("gdn", False), ("kda", True)):
        m = Model(gate=gate, v_first=v_first)
        ctx = m.context(1, 1)
        gen = torch.Generator(device="cuda").manual_seed(5)
        n, S = 7, 3
        q = torch.randn((n, m.G * m.H, m.d), generator=gen, device="cuda").bfloat16()
        k, v = ((torch.randn((n, m.H, m.d), generator=gen, device="cuda") / 12).bfloat16() for _ in range(2))
        beta, g = gates(m, (n,))
        slots = torch.tensor([2, 0, 2, 2, 0, 1, 2], dtype=torch.int32, device="cuda")
        a = torch.randn((S, m.H, m.d, m.d), generator=gen, device="cuda")
        b, oa, ob = a.clone(), torch.empty_like(q), torch.empty_like(q)
        ctx.delta_step(q, k, v, beta, g, a, oa, slots=slots)
        for i in range(n):
            one = [t[i:i + 1].clone() for t in (q, k, v, beta, g)]     # rows of their own: 16-byte aligned
            ctx.delta_step(*one, b, ob[i:i + 1], slots=slots[i:i + 1])
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(oa, ob)


def test_training_ends_gradients():
    """Embedding -> layer norm -> product, and back to the table, with the residual stream's gradient: against
    the same chain in 64 bits."""
    V, D, N, n = 50, 264, 136, 300
    gen = torch.Generator().manual_seed(3)

    def randn(*s):
        return torch.randn(s, generator=gen)

    tok = torch.randint(-1, V, (n,), generator=gen).to(torch.int32)
    table, w, dy, dsum = randn(V, D).bfloat16(), (randn(N, D) / 16).bfloat16(), randn(n, N).bfloat16(), randn(n, D).bfloat16()
    nw, nb = 1 + 0.2 * randn(D), 0.1 * randn(D)
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    c = {k: v.cuda() for k, v in dict(tok=tok, table=table, w=w, dy=dy, dsum=dsum, nw=nw, nb=nb).items()}
    x, y = (torch.empty((n, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    z = torch.empty((n, N), dtype=torch.bfloat16, device="cuda")
    ctx.embed_fwd(c["tok"], c["table"], x, scale=2.0)
    ctx.layernorm_fwd(x, c["nw"], bias=c["nb"], y=y, eps=EPS)
    ctx.linear_fwd(y, c["w"], z)
    back = ctx.linear_bwd(y, c["w"], c["dy"])
    norm = ctx.layernorm_bwd(x, c["nw"], back["dx"], dsum=c["dsum"], eps=EPS)
    grad = ctx.embed_bwd(c["tok"], norm["ds"], torch.empty_like(c["table"]), scale=2.0)
    torch.cuda.synchronize()

    def r(a):
        return torch.from_numpy(np.ascontiguousarray(a)).bfloat16().double().numpy()

    t64 = table.double().numpy()
    x64 = r(np.where((tok.numpy() >= 0)[:, None], 2.0 * t64[np.maximum(tok.numpy(), 0)], 0.0))
    y64 = r(om.layernorm_forward(x64, nw, nb, EPS)["y"])
    b64 = ol.linear_backward(y64, w, dy)
    n64 = om.layernorm_backward(x64, nw, EPS, r(b64["dx"]), dsum)
    g64 = om.embed_backward(tok, r(n64["ds"]), V, 2.0)["dtable"]
    # roundings of bf16 tensors along the chain, each 2^-8 of a value at most: under four at any of these
    for got, ref in ((z, ol.linear_forward(y64, w)["z"]), (back["dw"], b64["dw"]), (norm["ds"], n64["ds"]),
                     (norm["dweight"], n64["dweight"]), (norm["dbias"], n64["dbias"]), (grad, g64)):
        got = got.double().cpu().numpy()
        assert np.linalg.norm(got - ref) <= 4 * 2.0 ** -8 * np.linalg.norm(ref)


def steps_of(ctx, seed, n=640, D=264, V=1000):
    """One pass through all steps over tensors of its own; the outputs."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rb(*s):
        return torch.randn(s, generator=gen, device="cuda").bfloat16()

    t = dict(tok=torch.randint(-1, V, (n,), generator=gen, device="cuda").to(torch.int32), table=rb(V, D), dy=rb(n, D),
             w=1 + 0.1 * torch.randn(D, generator=gen, device="cuda"), b=torch.randn(D, generator=gen, device="cuda"),
             x=rb(n, D), r=rb(n, D), cw=torch.randn((D, 4), generator=gen, device="cuda"),
             q=rb(9, 4, 128), k=rb(9, 2, 128) * 0.08, v=rb(9, 2, 128), beta=torch.rand((9, 2), generator=gen, device="cuda").bfloat16(),
             g=-torch.rand((9, 2), generator=gen, device="cuda"), state=torch.randn((6, 2, 128, 128), generator=gen, device="cuda"),
             win=rb(6, 3, D), slots=torch.tensor([5, 0, 5, -1, 2, 2, 3, 0, 1], dtype=torch.int32, device="cuda"))
    o = dict(e=rb(n, D), s=rb(n, D), y=rb(n, D), y8=rb(n, D).to(torch.float8_e4m3fn), sc=torch.zeros(n, device="cuda"),
             ds=rb(n, D), dw=torch.zeros(D, device="cuda"), db=torch.zeros(D, device="cuda"), dt=rb(V, D), o=rb(9, 4, 128),
             so=t["state"].clone(), cy=rb(9, D), wo=t["win"].clone())
    ws = torch.empty(max(ctx.layernorm_bwd_workspace_bytes(n, D), ctx.embed_bwd_workspace_bytes(n, V, D)),
                     dtype=torch.uint8, device="cuda")

    def go():
        ctx.embed_fwd(t["tok"], t["table"], o["e"], scale=3.0)
        ctx.layernorm_fwd(o["e"], t["w"], bias=t["b"], residual=t["r"], sum_out=o["s"], y=o["y"], y8=o["y8"], scale=o["sc"])
        ctx.layernorm_bwd(o["s"], t["w"], t["dy"], dsum=o["y"], out=dict(ds=o["ds"], dweight=o["dw"], dbias=o["db"]), workspace=ws)
        ctx.embed_bwd(t["tok"], o["ds"], o["dt"], scale=3.0, workspace=ws)
        ctx.conv1d_step(o["dt"][:9], t["cw"], None, t["win"], o["cy"], slots=t["slots"], state_out=o["wo"])
        ctx.delta_step(t["q"], t["k"], t["v"], t["beta"], t["g"], t["state"], o["o"], slots=t["slots"], state_out=o["so"])
        return o
    return t, go


def context():
    return cpdr.Context(1, 1, 2, 128, 1, dtype="bf16", Hq=4, conv_width=4)


def same(a, b):
    return all(torch.equal(a[k].view(torch.uint8) if a[k].dtype is torch.float8_e4m3fn else a[k],
                           b[k].view(torch.uint8) if b[k].dtype is torch.float8_e4m3fn else b[k]) for k in a)


def kept(o):
    return {k: v.clone() for k, v in o.items()}


def test_captured_and_replayed_over_changing_inputs():
    ctx = context()
    t, go = steps_of(ctx, 1)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go()
    for seed in (2, 3, 4):
        other, _ = steps_of(ctx, seed)
        for k in t:
            t[k].copy_(other[k])
        out["so"].copy_(t["state"])
        out["wo"].copy_(t["win"])
        want = kept(go())
        for v in out.values():
            v.view(torch.uint8).fill_(77) if v.dtype is torch.float8_e4m3fn else v.fill_(7)
        out["so"].copy_(t["state"])
        out["wo"].copy_(t["win"])
        out["cy"].copy_(want["cy"])       # rows without a slot are left as they were
        out["o"].copy_(want["o"])
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want)
    ctx.check_device_status()


def test_two_streams_at_once():
    """Calls of one context on two streams whose work overlaps, each with its own tensors and workspace."""
    ctx = context()
    runs = [steps_of(ctx, s, n=5000) for s in (5, 6)]
    ref = []
    for _, go in runs:
        go()
        torch.cuda.synchronize()
        ref.append(kept(go()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    outs = [None, None]
    for _ in range(6):
        for i, st in enumerate(streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                outs[i] = runs[i][1]()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(ref, outs))


def test_what_a_call_makes_belongs_to_the_stream_it_runs_on():
    """Gradients on a stream of their own, whose workspaces and outputs are made by the call, while the current
    stream keeps taking and filling memory."""
    ctx = context()
    gen = torch.Generator(device="cuda").manual_seed(11)
    n, D, V = 5000, 520, 400
    s, dy = (torch.randn((n, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    w, tok = torch.ones(D, device="cuda"), torch.randint(0, V, (n,), generator=gen, device="cuda").to(torch.int32)
    norm = ctx.layernorm_bwd(s, w, dy)
    table = ctx.embed_bwd(tok, dy, torch.empty((V, D), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tables = [torch.empty_like(table) for _ in range(8)]
    torch.cuda.synchronize()
    got = []
    for t in tables:
        got.append((ctx.layernorm_bwd(s, w, dy, stream=side), ctx.embed_bwd(tok, dy, t, stream=side)))
        for _ in range(4):
            torch.full((4 * n * D,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(a[k], norm[k]) for k in norm) and torch.equal(b, table)


def test_a_chain_of_calls_equals_the_calls_one_by_one():
    """Kernels may begin while the one before them ends: a chain over shared buffers and one workspace, against
    the same calls with a synchronisation after each."""
    ctx = context()
    _, go = steps_of(ctx, 21)

    def chain(wait):
        _, go = steps_of(ctx, 21)
        out = []
        for _ in range(10):
            out.append(kept(go()))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out

    real = {f: getattr(ctx, f) for f in ("embed_fwd", "layernorm_fwd", "layernorm_bwd", "embed_bwd", "conv1d_step", "delta_step")}

    def waiting(f):
        def call(*a, **k):
            r = f(*a, **k)
            torch.cuda.synchronize()
            return r
        return call

    free = chain(False)
    for f, call in real.items():
        setattr(ctx, f, waiting(call))
    for a, b in zip(free, chain(True)):
        assert same(a, b)
