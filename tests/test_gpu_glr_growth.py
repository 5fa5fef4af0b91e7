"""The gated linear recurrence where gates are positive: products of its
factors pass fp32's range although the states stay finite.  Zero and small
states under such gates, a gate of -infinity behind them, growth and decay in
turn, all against the fp64 oracle with its error bounds (oracle/layer_steps.py),
in every layout and type, forward and backward; and what one channel's growth
or NaN does to the others: nothing, to the last bit.
"""
import math

import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol
from test_gpu_glr import both, close, draw
from test_gpu_glr_gates import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,gate", [(2, 60.0), (12, 8.0), (40, 88.0), (512, 8.0), (5000, 3.0)])
def test_zero_stays_zero(T, gate, dtype):
    """Token by token everything is 0; a product of the factors is infinite."""
    inp = {k: torch.zeros_like(v) for k, v in draw(1, T, 72, 1, dtype, 1).items()}
    inp["g"] += gate
    for k, v in run(inp, dtype, h0=False, dhT=False).items():
        assert (v == 0).all(), k


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [13, 130, 1500])
def test_minus_infinity_behind_growth(T, dtype):
    """Twelve tokens of gate 8, whose factors' product overflows, then the state is dropped; every
    13 tokens again.  x is 0 but for the twelfth token, dy but for the first: no state passes e^8."""
    inp = draw(1, T, 72, 1, dtype, 2)
    at = torch.arange(T) % 13
    inp["g"][0, at < 12] = 8.0
    inp["g"][0, at == 12] = float("-inf")
    inp["x"][0, at != 11] = 0
    inp["dy"][0, at != 0] = 0
    inp["h0"].zero_()
    inp["dhT"].zero_()
    both(inp, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lo", [0.0, -30.0])
@pytest.mark.parametrize("B,T,C", [(1, 5, 8), (2, 100, 72), (1, 1100, 136), (1, 4500, 64)])
def test_growth_and_decay_in_turn(B, T, C, lo, dtype):
    """g_t = s_t - s_{t-1}, s_t in lo .. lo + 40: every product of factors lies within e^-40 .. e^40,
    but positive gates alone sum to hundreds in every group."""
    inp = draw(B, T, C, B, dtype, 3)
    gen = torch.Generator().manual_seed(T)
    s = lo + 40 * torch.rand((B, T + 1, C), generator=gen)
    inp["g"] = s[:, 1:] - s[:, :-1]
    both(inp, dtype)


def test_small_states_grow():
    """1e-30 through 50 tokens of gate 2 to 2.7e13, and back down; the same backward."""
    inp = draw(1, 240, 64, 1, "fp32", 4)
    g = torch.cat([torch.full((50,), 2.0), torch.full((50,), -2.0)])
    inp["g"] = g.repeat(3)[:240].reshape(1, 240, 1).expand(1, 240, 64).contiguous()
    for k in ("x", "dy"):
        inp[k].zero_()
    for k in ("h0", "dhT"):
        inp[k] *= 1e-30
    both(inp, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("first,second,back", [(0, 1, 2), (5, 20, 40), (3, 200, 1100)])
def test_states_that_only_the_initial_state_keeps_finite(first, second, back, dtype):
    """From -3e38, 3e38 twice and back: 0, 3e38, 0.  From zero the same terms would overflow."""
    inp = draw(1, 1200, 64, 1, dtype, 10)
    inp["g"].zero_()
    inp["x"].zero_()
    inp["x"][0, [first, second]] = 3e38
    inp["x"][0, back] = -3e38
    inp["h0"][:] = -inp["x"][0, first].float()
    inp["dy"].mul_(1e-6)
    inp["dhT"].mul_(1e-6)
    both(inp, dtype)


@pytest.mark.parametrize("gate", [0.06, 0.0625, 0.0626, 0.25])
def test_slow_growth_on_both_sides_of_the_rule(gate):
    """Sums of positive gates next to the one over 16 tokens where the kernels change over."""
    T = int(70 / gate)
    inp = draw(1, T, 72, 1, "fp32", 5)
    inp["g"] = torch.full((1, T, 72), gate)
    inp["g"][0, :, ::5] *= -1
    inp["g"][0, ::3, 1] = 0.0
    both(inp, "fp32")


def waves(T, C, gen):
    """Log gates whose products lie within e^-30 .. e^30 while positive ones sum to hundreds."""
    s = 30 * torch.rand((1, T + 1, C), generator=gen)
    return s[:, 1:] - s[:, :-1]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,R,lengths", [(320, 2, None), (1200, 3, [100, 0, 1, 699, 400]), (2320, 2, [2320])])
def test_zigzag_and_packed(T, R, lengths, dtype):
    cu = None if lengths is None else np.cumsum([0] + lengths).tolist()
    inp = draw(1, T, 40, 1 if lengths is None else len(lengths), dtype, 6)
    inp["g"] = waves(T, 40, torch.Generator().manual_seed(T))
    both(inp, dtype, cu=cu, R=R, zigzag=True)
    both(inp, dtype, cu=cu)


def test_one_growing_channel_among_others():
    """Growth now and then, in one channel: steps with and without it follow one another."""
    inp = draw(1, 4000, 64, 1, "bf16", 7)
    inp["g"][0, 700:720, 5] = 4.0
    inp["g"][0, 720, 5] = -80.0
    inp["g"][0, 2100:2104, 40] = 20.0
    inp["g"][0, 2104:2108, 40] = -20.0
    inp["g"][0, 3999, 63] = 3.0
    both(inp, "bf16")


@pytest.mark.parametrize("T", [50, 700, 3000])
def test_growth_and_nan_stay_in_their_channels(T):
    inp = draw(1, T, 72, 1, "bf16", 8)
    clean = {k: v.clone() for k, v in inp.items()}
    ref = run(inp, "bf16")
    inp["g"][0, T // 3, 10] = 70.0
    inp["g"][0, T // 3 + 1, 10] = -70.0
    inp["g"][0, T // 2, 33] = float("nan")
    got = run(inp, "bf16")
    others = [c for c in range(72) if c not in (10, 33)]
    for k in ref:
        assert torch.equal(ref[k][..., others], got[k][..., others]), k
    # the NaN's channel: from its token on all is NaN, before it the state is what it was (both
    # within the bound of the exact one); gradients the other way
    f, b = ol.glr_forward(clean["x"], clean["g"], clean["h0"]), \
        ol.glr_backward(clean["x"], clean["g"], clean["dy"], clean["h0"], clean["dhT"])
    close(got["y"][0, :T // 2, 33], f["y"][0, :T // 2, 33], f["e_y"][0, :T // 2, 33], "bf16")
    assert got["y"][0, T // 2:, 33].isnan().all() and got["hT"][0, 33].isnan()
    close(got["dx"][0, T // 2:, 33], b["dx"][0, T // 2:, 33], b["e_dx"][0, T // 2:, 33], "bf16")
    assert got["dx"][0, :T // 2, 33].isnan().all() and got["dh0"][0, 33].isnan()
    assert got["y"][..., 10].isfinite().all() and math.isfinite(got["hT"][0, 10])


def test_same_bits_from_a_graph():
    T = 1500
    inp = {k: v.cuda() for k, v in draw(1, T, 72, 1, "fp32", 9).items()}
    inp["g"] = waves(T, 72, torch.Generator().manual_seed(1)).cuda()
    ctx = cpdr.Context(1, T, 1, 64, 1, dtype="fp32")

    def go():
        y, hT = torch.empty_like(inp["x"]), torch.empty_like(inp["h0"])
        carry = torch.empty(ctx.glr_carry_shape(72), device="cuda")
        ctx.glr_fwd(inp["x"], inp["g"], y, h0=inp["h0"], hT=hT, carry=carry)
        return [y, hT, carry, *ctx.glr_bwd(inp["x"], inp["g"], carry, inp["dy"], dhT=inp["dhT"]).values()]

    ref = go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = go()
    for t in captured:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref, captured):
        assert torch.equal(a, b)
