"""The activations where they fall off: SiLU and GELU of z from far below zero,
and their derivatives, to a relative error (values of 1e-6 and less matter to
nothing but their own size).

z comes from the bias alone (x = 0), so it is exact in fp32.  Bars: half a step
of bf16 for what is rounded to it, and 2e-4 of the value: the polynomial's
6.4e-5, and the roundings of exp's argument, which is up to 126 in units of
log 2 and passes three products (126 ln 2 * 3 * 2^-24 = 1.6e-5), of the
quotient and of the products around them.
"""
import math

import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr

pytestmark = pytest.mark.gpu

REL = 2e-4
HALF = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def ctx(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    return cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")


def phi(z):
    """Phi(z) for z <= 0, by erfc (erf would cancel)."""
    return np.vectorize(lambda v: 0.5 * math.erfc(-v / math.sqrt(2)))(z)


@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("act,lo", [("gelu", -12.5), ("silu", -80.0)])
def test_values(ctx, rows, act, lo):
    N = 4096
    z = torch.linspace(lo, 0.0, N + 1)[:-1].contiguous()
    zero = dict(device="cuda", dtype=torch.bfloat16)
    y = torch.empty(rows, N, **zero)
    ctx.linear_fwd(torch.zeros(rows, 8, **zero), torch.zeros(N, 8, **zero), y, bias=z.cuda(), activation=act)
    z64 = z.double().numpy()
    ref = z64 * phi(z64) if act == "gelu" else z64 / (1 + np.exp(-z64))
    got = y.double().cpu().numpy()
    assert (got == got[0]).all()
    err = np.abs(got[0] / ref - 1)
    assert err.max() <= HALF + REL, (err.max(), z64[err.argmax()])


@pytest.mark.parametrize("act,lo", [("gelu", -12.5), ("silu", -80.0)])
def test_derivatives(ctx, act, lo):
    """dbias of one row of dy = 1: the derivative, in fp32."""
    N = 4096
    z = torch.linspace(lo, -3.0, N).bfloat16()
    bf = dict(device="cuda", dtype=torch.bfloat16)
    out = ctx.linear_bwd(torch.zeros(1, 8, **bf), torch.zeros(N, 8, **bf), torch.ones(1, N, **bf), z=z[None].cuda(),
                         activation=act, out=dict(dbias=torch.empty(N, device="cuda")))
    z64 = z.double().numpy()
    if act == "gelu":
        ref = phi(z64) + z64 * np.exp(-z64 * z64 / 2) / math.sqrt(2 * math.pi)
    else:
        s = 1 / (1 + np.exp(-z64))
        ref = s * (1 + z64 * (1 - s))
    err = np.abs(out["dbias"].double().cpu().numpy() / ref - 1)
    assert err.max() <= REL, (err.max(), z64[err.argmax()])


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_far_away(ctx, act):
    """Where nothing is left, and where the activation is the identity."""
    z = torch.tensor([-1e30, -500.0, -90.0, -0.0, 0.0, 40.0, 500.0, 1e30]).repeat(2)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    y = torch.empty(2, 16, **bf)
    ctx.linear_fwd(torch.zeros(2, 8, **bf), torch.zeros(16, 8, **bf), y, bias=z.cuda(), activation=act)
    assert (y[:, :5] == 0).all() and torch.equal(y[0, 5:8].cpu(), z[5:8].bfloat16())
