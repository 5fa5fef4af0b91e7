"""Layer norm where the blocks are persistent (rows of bf16 to e4m3 or without a
residual): more rows than one wave, the sum and both outputs of one call against
the fp64 oracle, and the in-place forms, whose later rows are on their way
while earlier ones are written."""
import numpy as np
import pytest
import torch

from oracle import layer_steps as ol
from oracle import model_steps as om
from test_gpu_layernorm import EPS, _cuda, close, context, draw  # noqa: F401  (_cuda: the GPU or a skip)

pytestmark = pytest.mark.gpu

# rows beyond what the blocks take at once: 8, 4, 2 rows a block and one, two blocks a multiprocessor
SHAPES = [(5003, 512), (2601, 1024), (1303, 2048), (1301, 1736), (701, 4096), (700, 4088)]


def outputs(x, scale=True):
    y8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    return y8, torch.full((len(x),), float("nan"), device="cuda") if scale else None


def same8(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("rows,width", SHAPES)
@pytest.mark.parametrize("res,bias", [("r", "b"), (None, None)])
def test_sum_and_both_outputs_of_one_call(rows, width, res, bias):
    d = draw(rows, width, "bf16", seed=13)
    c = {k: v.cuda() for k, v in d.items()}
    s, y = (torch.full_like(c["x"], float("nan")) for _ in range(2))
    y8, scale = outputs(s)
    context("bf16").layernorm_fwd(c["x"], c["w"], bias=c.get(bias), residual=c.get(res), sum_out=s, y=y, y8=y8, scale=scale,
                                  eps=EPS)
    torch.cuda.synchronize()
    f = om.layernorm_forward(d["x"], d["w"], d.get(bias), EPS, d.get(res))
    close(s, f["s"], 0, "bf16")
    close(y, f["y"], f["e_y"], "bf16")
    # the scale is as far off as the row's largest value may be, and a quotient's rounding; an 8-bit value by half
    # a step of e4m3 (2^-4, or 2^-10 of the scale below the normal range), the quotient's roundings and the scale's
    rs, sc = ol.e4m3_scale(f["y"]), scale.double().cpu().numpy()
    assert (np.abs(sc - rs) <= f["e_y"].max(axis=1) / 448 + 4 * ol.U32 * rs).all()
    got = y8.double().cpu().numpy() * sc[:, None]
    tol = (2.0 ** -4 + 8 * ol.U32) * np.abs(f["y"]) + 2.0 ** -10 * sc[:, None] + 2 * f["e_y"]
    tol += np.abs(f["y"]) * (np.abs(sc - rs) / rs)[:, None]
    assert (np.abs(got - f["y"]) <= tol).all()


@pytest.mark.parametrize("rows,width", SHAPES)
def test_in_place(rows, width):
    c = {k: v.cuda() for k, v in draw(rows, width, "bf16", seed=17).items()}
    ctx = context("bf16")
    kw = dict(bias=c["b"], eps=EPS)
    y = torch.empty_like(c["x"])
    y8, scale = outputs(y)
    ctx.layernorm_fwd(c["x"], c["w"], y=y, y8=y8, scale=scale, **kw)
    x = c["x"].clone()
    ctx.layernorm_fwd(x, c["w"], y=x, **kw)                       # y = x, without the 8-bit output and with it
    assert torch.equal(x, y)
    x, (z8, zs) = c["x"].clone(), outputs(y)
    ctx.layernorm_fwd(x, c["w"], y=x, y8=z8, scale=zs, **kw)
    assert torch.equal(x, y) and same8(z8, y8) and torch.equal(zs, scale)
    s = torch.empty_like(y)
    ctx.layernorm_fwd(c["x"], c["w"], residual=c["r"], sum_out=s, y=y, y8=y8, scale=scale, **kw)
    for name in ("x", "r"):                                        # sum_out = x or the residual, y the other one or neither
        for both in (False, True):
            t = {k: c[k].clone() for k in ("x", "r")}
            z8, zs = outputs(y)
            other = t["r" if name == "x" else "x"]
            ctx.layernorm_fwd(t["x"], c["w"], residual=t["r"], sum_out=t[name], y=other if both else None, y8=z8, scale=zs, **kw)
            assert torch.equal(t[name], s) and same8(z8, y8) and torch.equal(zs, scale)
            assert torch.equal(other, y if both else c["r" if name == "x" else "x"])
