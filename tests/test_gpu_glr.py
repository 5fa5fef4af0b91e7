"""GPU parity of the gated linear recurrence (cpdr_glr_fwd, _bwd, _step)
against the fp64 oracle (oracle/layer_steps.py), whose error bounds the
tolerances are, plus half a step of the output's type: one token to several
cluster steps, fixed-length rows, packed batches with empty sequences, the
zigzag layout, channels that fill no slice, gates of -infinity, initial and
final states in place, another stream, and a captured graph.
"""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol
from oracle import layout as olayout

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def draw(B, T, C, N, dtype, seed, slow=False):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16

    def randn(*s):
        return torch.randn(s, generator=gen)

    g = torch.log1p(-1e-3 * torch.rand((B, T, C), generator=gen)) if slow else \
        torch.nn.functional.logsigmoid(2.0 + 1.5 * randn(B, T, C))
    return dict(x=randn(B, T, C).to(dt), g=g, dy=randn(B, T, C).to(dt), h0=3 * randn(N, C), dhT=randn(N, C))


def close(got, ref, err, dtype):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    tol = err + ol.HALF_STEP[dtype] * (np.abs(ref) + err) + 1e-37
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / tol).max()))


def both(inp, dtype, cu=None, R=1, zigzag=False, h0=True, dhT=True):
    """Forward and backward on the GPU and in the oracle, in sequence order."""
    B, T, C = inp["x"].shape
    ctx = cpdr.Context(B, T, 1, 64, R, dtype=dtype, cu_seqlens=cu, layout="zigzag" if zigzag else "contiguous")
    to = (lambda t: olayout.to_zigzag(t, R).contiguous()) if zigzag else (lambda t: t)
    back = (lambda t: olayout.from_zigzag(t.cpu(), R)) if zigzag else (lambda t: t.cpu())
    d = {k: to(v).cuda() if v.dim() == 3 else v.cuda() for k, v in inp.items()}
    y = torch.full_like(d["x"], float("nan"))
    hT = torch.full_like(d["h0"], float("nan"))
    carry = torch.full(ctx.glr_carry_shape(C), float("nan"), device="cuda")
    ctx.glr_fwd(d["x"], d["g"], y, h0=d["h0"] if h0 else None, hT=hT, carry=carry)
    grads = {k: torch.full_like(d[s], float("nan")) for k, s in (("dx", "x"), ("dg", "g"), ("dh0", "h0"))}
    ctx.glr_bwd(d["x"], d["g"], carry, d["dy"], dhT=d["dhT"] if dhT else None, out=grads)
    torch.cuda.synchronize()
    hh, dd = (inp["h0"] if h0 else None), (inp["dhT"] if dhT else None)
    f = ol.glr_forward(inp["x"], inp["g"], hh, cu)
    b = ol.glr_backward(inp["x"], inp["g"], inp["dy"], hh, dd, cu)
    close(back(y), f["y"], f["e_y"], dtype)
    close(hT, f["hT"], f["e_hT"], "fp32")
    close(back(grads["dx"]), b["dx"], b["e_dx"], dtype)
    close(back(grads["dg"]), b["dg"], b["e_dg"], "fp32")
    close(grads["dh0"], b["dh0"], b["e_dh0"], "fp32")
    # the carry: the state before every 16th token, sequence after sequence
    at = np.concatenate([np.arange(s, e, 16) + bb * T for bb, s, e in ol.bounds_of(B, T, cu)] or [np.zeros(0, int)])
    prev, ep = f["prev"].reshape(B * T, C)[at.astype(int)], f["e_prev"].reshape(B * T, C)[at.astype(int)]
    close(carry, prev, ep, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,C", [(1, 1, 8), (1, 2, 64), (3, 15, 72), (1, 16, 136), (2, 17, 8), (1, 127, 64),
                                   (1, 129, 200), (2, 1023, 64), (1, 1025, 8), (1, 2500, 72), (5, 300, 1024)])
def test_fixed_length_rows(B, T, C, dtype):
    both(draw(B, T, C, B, dtype, 100 + T), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths", [[1], [1, 0, 1], [0, 33, 16, 0, 1500, 1, 130, 0], [2000, 3, 700], [7] * 40])
def test_packed(lengths, dtype):
    cu = np.cumsum([0] + lengths).tolist()
    both(draw(1, cu[-1], 72, len(lengths), dtype, 7), dtype, cu=cu)


@pytest.mark.parametrize("T,R,lengths", [(2, 1, None), (16, 8, None), (320, 2, None), (4 * 13 * 16, 8, None),
                                         (1200, 3, [100, 0, 1, 699, 400]), (2320, 2, [2320])])
def test_zigzag(T, R, lengths):
    cu = None if lengths is None else np.cumsum([0] + lengths).tolist()
    n = 2 if lengths is None else len(lengths)
    both(draw(2 if lengths is None else 1, T, 40, n, "bf16", 9), "bf16", cu=cu, R=R, zigzag=True)


def test_long_memory():
    """Gates next to 1: the state holds thousands of tokens."""
    both(draw(1, 6000, 8, 1, "fp32", 11, slow=True), "fp32")


def test_without_initial_and_final_gradients():
    both(draw(2, 200, 64, 2, "bf16", 13), "bf16", h0=False, dhT=False)


def test_minus_infinity_drops_the_state():
    inp = draw(1, 300, 64, 1, "fp32", 15)
    inp["g"][0, [0, 5, 130, 131, 299]] = float("-inf")
    inp["g"][0, 200, ::2] = float("-inf")
    both(inp, "fp32")


def test_many_channels_and_growing_gates():
    inp = draw(1, 70, 4104, 1, "bf16", 17)
    inp["g"][0, ::7] = 0.25                 # a > 1
    both(inp, "bf16")


def test_optional_outputs_and_states_in_place():
    inp = {k: v.cuda() for k, v in draw(2, 150, 64, 2, "bf16", 19).items()}
    ctx = cpdr.Context(2, 150, 1, 64, 1, dtype="bf16")
    y, y2 = torch.empty_like(inp["x"]), torch.empty_like(inp["x"])
    hT = torch.empty_like(inp["h0"])
    carry = torch.empty(ctx.glr_carry_shape(64), device="cuda")
    ctx.glr_fwd(inp["x"], inp["g"], y, h0=inp["h0"], hT=hT, carry=carry)
    state = inp["h0"].clone()
    ctx.glr_fwd(inp["x"], inp["g"], y2, h0=state, hT=state)
    assert torch.equal(y, y2) and torch.equal(state, hT)
    ref = ctx.glr_bwd(inp["x"], inp["g"], carry, inp["dy"], dhT=inp["dhT"])
    grad = inp["dhT"].clone()
    out = ctx.glr_bwd(inp["x"], inp["g"], carry, inp["dy"], dhT=grad,
                      out=dict(dx=torch.empty_like(y), dg=torch.empty_like(inp["g"]), dh0=grad))
    for k in ref:
        assert torch.equal(ref[k], out[k]), k
    none = ctx.glr_bwd(inp["x"], inp["g"], carry, inp["dy"], dhT=inp["dhT"],
                       out=dict(dx=torch.empty_like(y), dg=torch.empty_like(inp["g"]), dh0=None))
    assert torch.equal(none["dx"], ref["dx"])


def test_a_sequence_in_two_calls_equals_one():
    """hT of the first part as h0 of the second (to the bound of one fp32 path)."""
    inp = draw(1, 700, 64, 1, "fp32", 21)
    f = ol.glr_forward(inp["x"], inp["g"], inp["h0"])
    state = inp["h0"].cuda()
    ys = []
    for s, e in ((0, 333), (333, 334), (334, 700)):
        ctx = cpdr.Context(1, e - s, 1, 64, 1, dtype="fp32")
        x = inp["x"][:, s:e].contiguous().cuda()
        y = torch.empty_like(x)
        ctx.glr_fwd(x, inp["g"][:, s:e].contiguous().cuda(), y, h0=state, hT=state)
        ys.append(y)
    torch.cuda.synchronize()
    close(torch.cat(ys, 1), f["y"], f["e_y"], "fp32")
    close(state, f["hT"], f["e_hT"], "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,C,S", [(1, 8, 1), (5, 520, 9), (64, 1032, 70), (600, 64, 600)])
def test_step_over_slots(n, C, S, dtype):
    gen = torch.Generator().manual_seed(n)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    x = torch.randn((n, C), generator=gen).to(dt)
    g = torch.nn.functional.logsigmoid(2 + torch.randn((n, C), generator=gen))
    state = 2 * torch.randn((S, C), generator=gen)
    slots = torch.randperm(S, generator=gen)[:n].to(torch.int32)
    if n > 4:
        slots[1], slots[3], slots[n - 1] = -1, S, slots[0]     # padding, out of range, two tokens of one sequence
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype=dtype)
    ry, rs = ol.glr_steps(x, g, state, slots.tolist())
    y = torch.full((n, C), 7.0).to(dt).cuda()
    sd, out = state.cuda(), state.cuda()
    ctx.glr_step(x.cuda(), g.cuda(), sd, y, slots=slots.cuda(), state_out=out)
    inplace, y2 = state.cuda(), torch.full_like(y, 7.0)
    ctx.glr_step(x.cuda(), g.cuda(), inplace, y2, slots=slots.cuda())
    torch.cuda.synchronize()
    assert torch.equal(sd.cpu(), state)                        # the input is left alone
    assert torch.equal(out, inplace) and torch.equal(y, y2)
    untouched = sorted(set(range(S)) - set(slots.tolist()))
    assert torch.equal(out.cpu()[untouched], state[untouched])
    # at most two steps of STEP-sized roundings each
    close(out, rs, 2 * ol.STEP * (np.abs(rs) + 2 * np.abs(ol.as64(state)) + np.abs(ol.as64(x)).max()), "fp32")
    idle = np.isnan(ry)
    assert (y.cpu().double().numpy()[idle] == 7.0).all()
    ry, got = np.where(idle, 7.0, ry), y
    close(got, ry, 2 * ol.STEP * (np.abs(ry) + 2 * np.abs(ol.as64(state)).max() + np.abs(ol.as64(x)).max()), dtype)


def test_step_without_slots_equals_the_scan_of_one_token():
    n, C = 7, 264
    inp = draw(n, 1, C, n, "bf16", 23)
    d = {k: v.cuda() for k, v in inp.items()}
    ctx = cpdr.Context(n, 1, 1, 64, 1, dtype="bf16")
    y, hT = torch.empty_like(d["x"]), torch.empty_like(d["h0"])
    ctx.glr_fwd(d["x"], d["g"], y, h0=d["h0"], hT=hT)
    state = d["h0"].clone()
    y1 = torch.empty_like(d["x"][:, 0])
    ctx.glr_step(d["x"][:, 0].contiguous(), d["g"][:, 0].contiguous(), state, y1)
    torch.cuda.synchronize()
    f = ol.glr_forward(inp["x"], inp["g"], inp["h0"])
    close(state, f["hT"], f["e_hT"], "fp32")
    close(hT, f["hT"], f["e_hT"], "fp32")
    close(y1, f["y"][:, 0], f["e_y"][:, 0], "bf16")


def test_same_bits_on_another_stream_and_from_a_graph():
    inp = {k: v.cuda() for k, v in draw(1, 3000, 264, 1, "bf16", 25).items()}
    ctx = cpdr.Context(1, 3000, 1, 64, 1, dtype="bf16")

    def go():
        y, hT = torch.empty_like(inp["x"]), torch.empty_like(inp["h0"])
        carry = torch.empty(ctx.glr_carry_shape(264), device="cuda")
        ctx.glr_fwd(inp["x"], inp["g"], y, h0=inp["h0"], hT=hT, carry=carry)
        return [y, hT, carry, *ctx.glr_bwd(inp["x"], inp["g"], carry, inp["dy"], dhT=inp["dhT"]).values()]

    ref = go()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        other = go()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = go()
    for t in captured:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(ref, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    ctx = cpdr.Context(1, 64, 1, 64, 1, dtype="bf16")
    x = torch.zeros(1, 64, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(1, 64, 64, device="cuda")
    y = torch.empty_like(x)

    def refused(call, text):
        with pytest.raises(cpdr.CpdrError, match=text) as ei:
            call()
        assert ei.value.status == cpdr.ERR_INVALID

    refused(lambda: ctx.glr_fwd(x, g, x), "y overlaps x")
    refused(lambda: ctx.glr_fwd(x[..., :12].contiguous(), g[..., :12].contiguous(), y[..., :12].contiguous()),
            "multiple of 8")
    flat = torch.zeros(1, 64 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    refused(lambda: ctx.glr_fwd(flat[:, 1:4097].view(1, 64, 64), g, y), "16-byte aligned: x")
    h = torch.zeros(2, 64, device="cuda")
    refused(lambda: ctx.glr_step(x[0], g[0], h, y[0], slots=None), "at most num_slots")
    refused(lambda: ctx.glr_step(x[0, :1], g[0, :1], h, x[0, :1], slots=torch.zeros(1, dtype=torch.int32, device="cuda")),
            "y overlaps x")
    with pytest.raises(ValueError):
        ctx.glr_fwd(x, g, y, h0=torch.zeros(2, 64, device="cuda"))
    with pytest.raises(ValueError):
        ctx.glr_fwd(x.transpose(1, 2), g, y)
