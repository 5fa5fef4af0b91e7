"""GPU parity of the mixers' token steps (cpdr_delta_step, cpdr_conv1d_step)
against the fp64 oracle (oracle/model_steps.py): both gates, dtypes, head dims
and state layouts, grouped query heads, drafted tokens in mixed order, empty
rows, in-place and separate states, and their refusals.

Bars: the oracle's error bounds (a value dim's column of a state in its
2-norm) plus half a step of the output's type.
"""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol
from oracle import model_steps as om

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def draw_delta(n, H, G, d, gate, dtype, S, seed=0):
    gen = torch.Generator().manual_seed(1000 * n + 10 * H + seed)

    def randn(*s):
        return torch.randn(s, generator=gen)

    def unit(*s):
        t = randn(*s)
        return t / t.norm(dim=-1, keepdim=True)

    dt = DT[dtype]
    return dict(q=unit(n, H * G, d).to(dt), k=unit(n, H, d).to(dt), v=randn(n, H, d).to(dt),
                beta=torch.sigmoid(randn(n, H)).to(dt),
                g=torch.nn.functional.logsigmoid(2 + randn(n, H, *([d] if gate == "kda" else []))),
                state=0.3 * randn(S, H, d, d))


def run_delta(case, slots, dtype, gate, vfirst, scale=0.25, in_place=True, G=1):
    n, H, d = case["k"].shape
    ctx = cpdr.Context(1, 1, H, d, 1, gate=gate, dtype=dtype, scale=scale, Hq=H * G, state_v_first=vfirst)
    c = {k: t.cuda() for k, t in case.items()}
    state = c["state"].transpose(2, 3).contiguous() if vfirst else c["state"].clone()
    before = state.clone()
    out = state if in_place else torch.full_like(state, 99.0)
    o = torch.full((n, H * G, d), 7.0, device="cuda").to(DT[dtype])
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    ctx.delta_step(c["q"], c["k"], c["v"], c["beta"], c["g"], state, o, slots=sl, state_out=None if in_place else out)
    torch.cuda.synchronize()
    ctx.check_device_status()
    if not in_place:
        assert torch.equal(state, before)
    return o, out.transpose(2, 3) if vfirst else out


def check_delta(case, slots, o, out, dtype, scale=0.25, fill=None):
    listed = list(range(len(case["k"]))) if slots is None else slots
    r = om.delta_steps(case["q"], case["k"], case["v"], case["beta"], case["g"], case["state"], listed, scale)
    S = case["state"].shape[0]
    o, out = o.double().cpu().numpy(), out.double().cpu().numpy()
    live = np.array([0 <= s < S for s in listed], dtype=bool)
    assert (o[~live] == 7.0).all()
    tol = r["e_o"][live] + ol.HALF_STEP[dtype] * (np.abs(r["o"][live]) + r["e_o"][live]) + 1e-30
    err = np.abs(o[live] - r["o"][live])
    assert (err <= tol).all(), float(np.nanmax(err / tol))
    used = sorted({s for s in listed if 0 <= s < S})
    off = np.linalg.norm(out[used] - r["state"][used], axis=2)      # over the key dims
    assert (off <= r["e_state"][used] + 1e-30).all(), float(np.nanmax(off / (r["e_state"][used] + 1e-30)))
    rest = [s for s in range(S) if s not in used]
    want = case["state"].double().numpy()[rest] if fill is None else fill
    assert (out[rest] == want).all()


@pytest.mark.parametrize("vfirst", [False, True])
@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_token_each(dtype, d, gate, vfirst):
    case = draw_delta(5, 3, 1, d, gate, dtype, 9)
    slots = [8, 0, -1, 3, 9]          # an empty row and one past the pool
    o, out = run_delta(case, slots, dtype, gate, vfirst)
    check_delta(case, slots, o, out, dtype)


@pytest.mark.parametrize("vfirst", [False, True])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8])
def test_grouped_query_heads(G, vfirst):
    for dtype, d, gate in (("bf16", 128, "gdn"), ("fp32", 64, "kda")):
        case = draw_delta(4, 2, G, d, gate, dtype, 4, seed=G)
        slots = [2, 0, 2, 1]
        o, out = run_delta(case, slots, dtype, gate, vfirst, G=G)
        check_delta(case, slots, o, out, dtype)


MIXED = [
    [0, 0, 0, 0, 0],
    [2, 1, 2, -1, 1, 2, 0],
    [3] * 33 + [1],                                  # runs past a window of 32 rows
    [1] + [-1] * 40 + [1] + [5] * 70 + [1],          # a sequence's tokens far apart
    list(range(64)) * 2 + [63],
    [i % 3 for i in range(100)],
]


@pytest.mark.parametrize("vfirst", [False, True])
@pytest.mark.parametrize("slots", MIXED, ids=[str(i) for i in range(len(MIXED))])
def test_drafted_tokens(slots, vfirst):
    for dtype, gate, in_place in (("fp32", "gdn", True), ("bf16", "kda", False)):
        case = draw_delta(len(slots), 1, 2, 64, gate, dtype, max(slots) + 2, seed=len(slots))
        o, out = run_delta(case, slots, dtype, gate, vfirst, in_place=in_place, G=2)
        check_delta(case, slots, o, out, dtype, fill=None if in_place else 99.0)


@pytest.mark.parametrize("vfirst", [False, True])
def test_without_slots_row_i_is_slot_i(vfirst):
    case = draw_delta(3, 2, 1, 128, "gdn", "bf16", 5)
    o, out = run_delta(case, None, "bf16", "gdn", vfirst)
    check_delta(case, None, o, out, "bf16")


@pytest.mark.parametrize("vfirst", [False, True])
def test_gates_that_drop_and_grow(vfirst):
    """exp(-inf) = 0 drops the state, one key dim of it with the per-dim gate; positive gates let it grow."""
    for gate in ("gdn", "kda"):
        case = draw_delta(4, 1, 1, 64, gate, "fp32", 4, seed=3)
        case["g"][0] = -float("inf")
        case["g"][1].view(-1)[0] = -float("inf")
        case["g"][2] = 0.5
        case["g"][3] = -200.0
        o, out = run_delta(case, [0, 1, 2, 3], "fp32", gate, vfirst)
        check_delta(case, [0, 1, 2, 3], o, out, "fp32")


@pytest.mark.parametrize("vfirst", [False, True])
def test_one_state_does_not_reach_another(vfirst):
    """A slot of NaN and infinities, and rows of no slot that hold them, leave every other row alone."""
    case = draw_delta(4, 2, 1, 128, "gdn", "bf16", 6)
    slots = [5, -1, 2, 0]
    clean_o, clean = run_delta(case, slots, "bf16", "gdn", vfirst)
    for name in ("q", "k", "v", "beta", "g"):
        case[name][1] = float("nan")
    case["state"][5] = float("inf")
    case["state"][1] = float("nan")
    o, out = run_delta(case, slots, "bf16", "gdn", vfirst)
    assert torch.equal(o[[1, 2, 3]], clean_o[[1, 2, 3]]) and torch.equal(out[[0, 2, 3, 4]], clean[[0, 2, 3, 4]])
    assert out[1].isnan().all() and not o[0].isfinite().any()


def test_many_rows():
    """65535 rows, most of them empty: the longest list of rows; its one sequence's tokens lie at both ends."""
    n = 65535
    gen = torch.Generator().manual_seed(5)
    at = [0, 7, 40000, n - 1]
    slots = torch.full((n,), -1, dtype=torch.int32)
    slots[at] = torch.tensor([1, 0, 1, 1], dtype=torch.int32)
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="fp32", scale=0.25)
    rows = draw_delta(4, 1, 1, 64, "gdn", "fp32", 2)
    c = {}
    for name in ("q", "k", "v", "beta", "g"):
        c[name] = torch.randn((n, *rows[name].shape[1:]), generator=gen)
        c[name][at] = rows[name]
        c[name] = c[name].cuda()
    state, o = rows["state"].cuda(), torch.full((n, 1, 64), 7.0, device="cuda")
    ctx.delta_step(c["q"], c["k"], c["v"], c["beta"], c["g"], state, o, slots=slots.cuda())
    torch.cuda.synchronize()
    check_delta(rows, [1, 0, 1, 1], o[at], state, "fp32")
    rest = torch.ones(n, dtype=torch.bool)
    rest[at] = False
    assert (o.cpu()[rest] == 7.0).all()


def test_a_pool_past_2_31_elements():
    """Slots whose offset passes 32 bits (a pool of 8.7 GB); the first and the last one are used."""
    S, H, d = 2 ** 31 // (8 * 128 * 128) + 200, 8, 128
    case = draw_delta(3, H, 1, d, "gdn", "bf16", 3)
    pool = torch.zeros((S, H, d, d), device="cuda")
    at = [S - 1, 0, 2 ** 31 // (H * d * d)]
    pool[at] = case["state"].cuda()
    ctx = cpdr.Context(1, 1, H, d, 1, dtype="bf16", scale=0.25)
    c = {k: t.cuda() for k, t in case.items()}
    o = torch.full((3, H, d), 7.0, device="cuda").bfloat16()
    ctx.delta_step(c["q"], c["k"], c["v"], c["beta"], c["g"], pool, o,
                   slots=torch.tensor(at, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    check_delta(case, [0, 1, 2], o, pool[at], "bf16")


def test_delta_refusals():
    case = {k: t.cuda() for k, t in draw_delta(3, 2, 1, 64, "gdn", "bf16", 4).items()}
    ctx = cpdr.Context(1, 1, 2, 64, 1, dtype="bf16")
    a = (case["q"], case["k"], case["v"], case["beta"], case["g"])
    o = torch.empty_like(case["q"])
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(cpdr.CpdrError, match="at most num_slots"):
        ctx.delta_step(*a, case["state"][:2], o)
    with pytest.raises(cpdr.CpdrError, match="overlaps"):
        ctx.delta_step(*a, case["state"], case["v"], slots=slots)
    with pytest.raises(cpdr.CpdrError, match="overlaps"):
        ctx.delta_step(*a, case["state"][:3], o, slots=slots, state_out=case["state"][1:])
    with pytest.raises(cpdr.CpdrError, match="num_slots must be positive"):
        ctx.delta_step(*a, case["state"][:0], o, slots=slots)
    with pytest.raises(ValueError, match="g must be"):
        ctx.delta_step(*a[:4], case["g"][..., None].expand(3, 2, 64).contiguous(), case["state"], o, slots=slots)
    with pytest.raises(ValueError, match="slots must be"):
        ctx.delta_step(*a, case["state"], o, slots=slots.long())
    with pytest.raises(ValueError, match="o must be"):
        ctx.delta_step(*a, case["state"], o[:, :1], slots=slots)
    lib, p = ctx._lib, lambda t: t.data_ptr()   # noqa: E731
    args = [ctx._h, *(p(t) for t in a), p(case["state"]), p(case["state"]), p(slots)]
    for n, S, want in ((-1, 4, "n must be"), (65536, 4, "n must be")):
        assert lib.cpdr_delta_step(*args, n, S, p(o), None) == cpdr.ERR_INVALID
        assert want in lib.cpdr_last_error().decode()
    for i in range(1, 8):
        broken = list(args)
        broken[i] = None
        assert lib.cpdr_delta_step(*broken, 3, 4, p(o), None) == cpdr.ERR_INVALID
        broken[i] = args[i] + 4
        assert lib.cpdr_delta_step(*broken, 3, 4, p(o), None) == cpdr.ERR_INVALID
        assert "aligned" in lib.cpdr_last_error().decode()
    assert lib.cpdr_delta_step(*args[:8], args[8] + 2, 3, 4, p(o), None) == cpdr.ERR_INVALID
    # no rows: nothing to do, whatever the tensors are
    assert lib.cpdr_delta_step(ctx._h, *([None] * 8), 0, 1, None, None) == cpdr.OK


# ------------------------------------------------------------------ conv
def conv_case(n, C, W, S, dtype, seed=0):
    gen = torch.Generator().manual_seed(100 * n + C + W + seed)
    return dict(x=torch.randn((n, C), generator=gen).to(DT[dtype]), w=torch.randn((C, W), generator=gen) / W ** 0.5,
                b=0.3 * torch.randn(C, generator=gen), state=torch.randn((S, W - 1, C), generator=gen).to(DT[dtype]))


def check_conv(case, slots, dtype, act="silu", bias=True, in_place=True):
    W, C, n = case["w"].shape[1], case["w"].shape[0], len(case["x"])
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype=dtype, conv_width=W)
    c = {k: t.cuda() for k, t in case.items()}
    state = c["state"].clone()
    out = state if in_place else torch.full_like(state, 9.0)
    y = torch.full((n, C), 7.0, device="cuda").to(DT[dtype])
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    ctx.conv1d_step(c["x"], c["w"], c["b"] if bias else None, state, y, slots=sl,
                    state_out=None if in_place else out, activation=act)
    torch.cuda.synchronize()
    listed = list(range(n)) if slots is None else slots
    r = om.conv_steps(case["x"], case["w"], case["b"] if bias else None, case["state"], listed, act)
    S = case["state"].shape[0]
    live = np.array([0 <= s < S for s in listed], dtype=bool)
    y = y.double().cpu().numpy()
    assert (y[~live] == 7.0).all()
    tol = r["e_y"][live] + ol.HALF_STEP[dtype] * (np.abs(r["y"][live]) + r["e_y"][live])
    assert (np.abs(y[live] - r["y"][live]) <= tol).all()
    used = sorted({s for s in listed if 0 <= s < S})
    want = case["state"].double().numpy() if in_place else np.full(case["state"].shape, 9.0)
    want[used] = r["state"][used]
    assert (out.double().cpu().numpy() == want).all()     # inputs are moved, not computed


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 6, 7, 8])
def test_conv_widths(W, dtype):
    for C, act, bias in ((8, "silu", True), (264, None, False), (1032, "silu", False)):
        check_conv(conv_case(5, C, W, 6, dtype), [4, -1, 0, 5, 6], dtype, act, bias)


@pytest.mark.parametrize("slots", MIXED, ids=[str(i) for i in range(len(MIXED))])
def test_conv_drafted_tokens(slots):
    for dtype, in_place in (("bf16", True), ("fp32", False)):
        check_conv(conv_case(len(slots), 40, 4, max(slots) + 2, dtype), slots, dtype, in_place=in_place)


def test_conv_without_slots():
    check_conv(conv_case(6, 2056, 4, 7, "bf16"), None, "bf16")


def test_conv_tokens_equal_the_conv_over_the_sequence():
    """A sequence's tokens one by one, from a window of zeros, give the conv over the sequence, to the bit."""
    T, C, W = 37, 1032, 4
    case = conv_case(T, C, W, 1, "bf16", seed=2)
    c = {k: t.cuda() for k, t in case.items()}
    ctx = cpdr.Context(1, T, 1, 64, 1, dtype="bf16", conv_width=W)
    want = torch.empty((1, T, C), dtype=torch.bfloat16, device="cuda")
    ctx.conv1d_fwd(c["x"][None], c["w"], c["b"], want)
    state = torch.zeros((1, W - 1, C), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    for t in range(20):
        ctx.conv1d_step(c["x"][t:t + 1], c["w"], c["b"], state, y[t:t + 1])
    ctx.conv1d_step(c["x"][20:], c["w"], c["b"], state, y[20:], slots=torch.zeros(T - 20, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(state[0], c["x"][T - 3:])


def test_conv_refusals():
    c = {k: t.cuda() for k, t in conv_case(3, 16, 4, 3, "bf16").items()}
    y = torch.empty_like(c["x"])
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16", conv_width=4)
    none = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    with pytest.raises((cpdr.CpdrError, ValueError)):
        none.conv1d_step(c["x"], c["w"], None, c["state"], y)
    with pytest.raises(cpdr.CpdrError, match="at most num_slots"):
        ctx.conv1d_step(c["x"], c["w"], None, c["state"][:2], y)
    with pytest.raises(cpdr.CpdrError, match="overlaps"):
        ctx.conv1d_step(c["x"], c["w"], None, c["state"], c["x"])
    with pytest.raises(cpdr.CpdrError, match="multiple of 8"):
        odd = c["x"][:, :12].contiguous()
        ctx.conv1d_step(odd, c["w"][:12].contiguous(), None, c["state"][..., :12].contiguous(), torch.empty_like(odd))
    with pytest.raises(KeyError):
        ctx.conv1d_step(c["x"], c["w"], None, c["state"], y, activation="gelu")
    lib, p = ctx._lib, lambda t: t.data_ptr()   # noqa: E731
    for act in (-1, 2):
        assert lib.cpdr_conv1d_step(ctx._h, p(c["x"]), p(c["w"]), None, p(c["state"]), p(c["state"]), None, 3, 3, 16,
                                    act, p(y), None) == cpdr.ERR_INVALID
    assert none._lib.cpdr_conv1d_step(none._h, p(c["x"]), p(c["w"]), None, p(c["state"]), p(c["state"]), None, 3, 3, 16,
                                      1, p(y), None) == cpdr.ERR_INVALID
