"""The factors exp(gate) of the gated linear recurrence: their accuracy over
the whole range of gates, and that a channel's results do not depend on the
gates of the channels beside it, to the last bit.
"""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol
from test_gpu_glr import draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def run(inp, dtype, h0=True, dhT=True):
    """Every output of a forward and a backward on the GPU."""
    B, T, C = inp["x"].shape
    ctx = cpdr.Context(B, T, 1, 64, 1, dtype=dtype)
    d = {k: v.cuda() for k, v in inp.items()}
    y = torch.full_like(d["x"], float("nan"))
    hT = torch.full_like(d["h0"], float("nan"))
    carry = torch.full(ctx.glr_carry_shape(C), float("nan"), device="cuda")
    ctx.glr_fwd(d["x"], d["g"], y, h0=d["h0"] if h0 else None, hT=hT, carry=carry)
    grads = ctx.glr_bwd(d["x"], d["g"], carry, d["dy"], dhT=d["dhT"] if dhT else None)
    torch.cuda.synchronize()
    ctx.check_device_status()
    return dict(y=y, hT=hT, carry=carry, **grads)


# One token from a state of 1 gives the factor itself.  Two units in the last
# place (4 U32) for the power of two, one rounding (U32) for the product that
# corrects its argument, and one to spare for the argument's own correction.
FACTOR = 6 * ol.U32


@pytest.mark.parametrize("lo,hi", [(-87.3, -30.0), (-30.0, -0.25), (-0.26, 0.26), (0.25, 30.0), (30.0, 88.0)])
def test_factor_over_the_range_of_gates(lo, hi):
    C = 8192
    g = torch.linspace(lo, hi, C)[None, None]
    zero = torch.zeros(1, 1, C)
    out = run(dict(x=zero, g=g, dy=zero, h0=torch.ones(1, C), dhT=torch.ones(1, C)), "fp32")
    ref = np.exp(g.double().numpy()[0])
    for k in ("hT", "dh0"):
        err = np.abs(out[k].double().cpu().numpy() / ref - 1)
        assert err.max() <= FACTOR, (k, err.max() / ol.U32, g[0, 0, int(err.argmax())])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [7, 100, 2500])
def test_bits_of_a_channel_do_not_depend_on_its_neighbours(T, dtype):
    """Slow channels (a memory of thousands of tokens) beside slow ones, beside
    fast ones, and beside one that is reset."""
    inp = draw(1, T, 72, 1, dtype, 31, slow=True)
    ref = run(inp, dtype)
    fast = torch.arange(72) % 5 == 3
    inp["g"][..., fast] = -2.0
    inp["g"][0, T // 2:, 3] = float("-inf")
    got = run(inp, dtype)
    for k in ref:
        assert torch.equal(ref[k][..., ~fast], got[k][..., ~fast]), k


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_bits_of_a_channel_do_not_depend_on_its_own_other_tokens(dtype):
    """A factor is a function of its gate alone: tokens in front of a reset leave no trace behind it."""
    inp = draw(1, 48, 64, 1, dtype, 33, slow=True)
    inp["g"][0, 20] = float("-inf")
    ref = run(inp, dtype)
    inp["g"][0, :20] = -3.0
    got = run(inp, dtype)
    for k in ("y", "hT"):
        tail = slice(20, None) if k == "y" else slice(None)
        assert torch.equal(ref[k][0, tail], got[k][0, tail]), k
