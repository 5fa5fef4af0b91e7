"""GPU parity of the layer norm (cpdr_layernorm_fwd, _bwd) against the fp64
oracle (oracle/model_steps.py): every group size's widths, odd row counts, both
dtypes, the residual's sum, large means, 8-bit outputs with their scales,
in-place forms, missing biases, NaN and infinities.

Bars: the oracle's error bounds plus half a step of the output's type; e4m3
values within half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below
the normal range) of the unrounded quotient.
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


def context(dtype):
    return cpdr.Context(1, 1, 1, 64, 1, dtype=dtype)


def draw(rows, width, dtype, seed=0, mean=1.0):
    gen = torch.Generator().manual_seed(1000 * width + rows + seed)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16

    def randn(*s):
        return torch.randn(s, generator=gen)

    return dict(x=(randn(rows, width) * torch.exp(randn(rows, 1)) + mean * randn(rows, 1)).to(dt),
                r=randn(rows, width).to(dt), dy=(randn(rows, width) + 0.5).to(dt), dsum=randn(rows, width).to(dt),
                w=1 + 0.3 * randn(width), b=0.3 * randn(width))


def close(got, ref, err, dtype):
    got = got.double().cpu().numpy()
    tol = err + ol.HALF_STEP[dtype] * (np.abs(ref) + err) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)))


def check(rows, width, dtype, seed=0, mean=1.0, eps=EPS):
    d = draw(rows, width, dtype, seed, mean)
    c = {k: v.cuda() for k, v in d.items()}
    ctx = context(dtype)
    for res, bias in ((None, "b"), ("r", None), ("r", "b")):
        f = om.layernorm_forward(d["x"], d["w"], d.get(bias), eps, d.get(res))
        s, y, y2 = (torch.full_like(c["x"], float("nan")) for _ in range(3))
        y8 = torch.empty((rows, width), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.full((rows,), float("nan"), device="cuda")
        kw = dict(residual=c.get(res), bias=c.get(bias), eps=eps)
        ctx.layernorm_fwd(c["x"], c["w"], sum_out=s, y=y, **kw)
        ctx.layernorm_fwd(c["x"], c["w"], y=y2, y8=y8, scale=scale, **kw)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
        close(s, f["s"], 0, dtype)
        close(y, f["y"], f["e_y"], dtype)
        # the scale is as far off as the row's largest value may be, and a quotient's rounding
        rs, sc = ol.e4m3_scale(f["y"]), scale.double().cpu().numpy()
        assert (np.abs(sc - rs) <= f["e_y"].max(axis=1) / 448 + 4 * ol.U32 * rs).all()
        got = y8.double().cpu().numpy() * sc[:, None]
        tol = (2.0 ** -4 + 8 * ol.U32) * np.abs(f["y"]) + 2.0 ** -10 * sc[:, None] + 2 * f["e_y"]
        tol += np.abs(f["y"]) * (np.abs(sc - rs) / rs)[:, None]
        assert (np.abs(got - f["y"]) <= tol).all()
    for dsum, bias in ((None, True), ("dsum", True), ("dsum", False)):
        b = om.layernorm_backward(d["x"], d["w"], eps, d["dy"], d.get(dsum))
        out = None if bias else dict(ds=torch.empty_like(c["x"]), dweight=torch.empty_like(c["w"]))
        out = ctx.layernorm_bwd(c["x"], c["w"], c["dy"], dsum=c.get(dsum), eps=eps, out=out)
        torch.cuda.synchronize()
        close(out["ds"], b["ds"], b["e_ds"], dtype)
        close(out["dweight"], b["dweight"], b["e_dweight"], "fp32")
        if bias:
            close(out["dbias"], b["dbias"], b["e_dbias"], "fp32")


WIDTHS = [8, 16, 24, 32, 40, 56, 64, 72, 96, 128, 136, 192, 256, 264, 384, 512, 520, 776, 1024, 1032, 1536, 2048, 2056,
          4096, 4104, 5208, 6144, 8192, 8200, 10000, 12288, 12296, 16376, 16384]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    check(37, width, dtype)


@pytest.mark.parametrize("rows,width", [(1, 8), (1, 64), (2, 2048), (3, 128), (15, 8), (16, 128), (17, 128), (3001, 128),
                                        (2049, 264), (700, 2048), (5, 16384)])
def test_rows(rows, width):
    check(rows, width, "bf16", seed=5)
    check(rows, width, "fp32", seed=6)


@pytest.mark.parametrize("width", [64, 776, 2048, 8192])
def test_large_means(width):
    """Rows whose mean is thousands of times their spread: the variance is that of the differences."""
    check(9, width, "fp32", seed=7, mean=3000.0)


def test_eps_of_zero():
    for rows, width in ((1, 8), (3, 64), (37, 136), (700, 264), (5, 776)):
        check(rows, width, "fp32", seed=11, eps=0.0)


def test_rows_without_variance():
    """Equal values: the norm is the bias, the gradient passes through 1 / sqrt(eps) alone."""
    for dtype in ("bf16", "fp32"):
        for value in (0.0, 3.140625, -1000.0, 1e4):
            d = draw(4, 264, dtype)
            d["x"][:] = value
            c = {k: v.cuda() for k, v in d.items()}
            y = torch.empty_like(c["x"])
            ctx = context(dtype)
            ctx.layernorm_fwd(c["x"], c["w"], bias=c["b"], y=y, eps=EPS)
            out = ctx.layernorm_bwd(c["x"], c["w"], c["dy"], eps=EPS)
            torch.cuda.synchronize()
            f, b = om.layernorm_forward(d["x"], d["w"], d["b"], EPS), om.layernorm_backward(d["x"], d["w"], EPS, d["dy"])
            close(y, f["y"], f["e_y"], dtype)
            close(out["ds"], b["ds"], b["e_ds"], dtype)


@pytest.mark.parametrize("width", [64, 2048, 8200])
def test_in_place(width):
    for dtype in ("bf16", "fp32"):
        d = draw(21, width, dtype, 3)
        c = {k: v.cuda() for k, v in d.items()}
        ctx = context(dtype)
        s, y = torch.empty_like(c["x"]), torch.empty_like(c["x"])
        kw = dict(bias=c["b"], eps=EPS)
        ctx.layernorm_fwd(c["x"], c["w"], residual=c["r"], sum_out=s, y=y, **kw)
        x, r = c["x"].clone(), c["r"].clone()
        ctx.layernorm_fwd(x, c["w"], residual=r, sum_out=r, y=x, **kw)
        assert torch.equal(x, y) and torch.equal(r, s)
        x, r = c["x"].clone(), c["r"].clone()
        ctx.layernorm_fwd(x, c["w"], residual=r, sum_out=x, y=r, **kw)
        assert torch.equal(r, y) and torch.equal(x, s)
        ref = ctx.layernorm_bwd(s, c["w"], c["dy"], dsum=c["dsum"], eps=EPS)
        for name in ("dy", "dsum"):
            t = {k: c[k].clone() for k in ("dy", "dsum")}
            out = ctx.layernorm_bwd(s, c["w"], t["dy"], dsum=t["dsum"], eps=EPS,
                                    out=dict(ds=t[name], dweight=torch.empty_like(c["w"]), dbias=torch.empty_like(c["w"])))
            assert all(torch.equal(out[k], ref[k]) for k in ref)


def test_nan_and_infinity_stay_in_their_rows():
    for dtype in ("bf16", "fp32"):
        for width in (24, 64, 2048, 8192):
            d = draw(40, width, dtype, 9)
            c = {k: v.cuda() for k, v in d.items()}
            ctx = context(dtype)
            clean = torch.empty_like(c["x"])
            ctx.layernorm_fwd(c["x"], c["w"], y=clean, eps=EPS)
            c["x"][5, 3], c["x"][17, width - 1] = float("nan"), float("inf")
            y, y8 = torch.empty_like(clean), torch.empty(clean.shape, dtype=torch.float8_e4m3fn, device="cuda")
            scale = torch.empty(40, device="cuda")
            ctx.layernorm_fwd(c["x"], c["w"], y=y, y8=y8, scale=scale, eps=EPS)
            torch.cuda.synchronize()
            ok = torch.ones(40, dtype=torch.bool)
            ok[[5, 17]] = False
            assert torch.equal(y[ok], clean[ok]) and scale[ok].isfinite().all()
            assert y[~ok].isnan().all() and scale[~ok].isnan().all()


def test_same_call_same_bits():
    d = {k: v.cuda() for k, v in draw(5001, 1360, "bf16").items()}
    ctx = context("bf16")
    ref = ctx.layernorm_bwd(d["x"], d["w"], d["dy"], dsum=d["dsum"])
    for _ in range(3):
        out = ctx.layernorm_bwd(d["x"], d["w"], d["dy"], dsum=d["dsum"])
        assert all(torch.equal(out[k], ref[k]) for k in ref)


def test_no_rows():
    ctx = context("bf16")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    ctx.layernorm_fwd(x, w, y=torch.empty_like(x))
    out = ctx.layernorm_bwd(x, w, x)
    torch.cuda.synchronize()
    assert (out["dweight"] == 0).all() and (out["dbias"] == 0).all()


def test_refusals():
    d = {k: v.cuda() for k, v in draw(4, 64, "bf16").items()}
    ctx = context("bf16")
    y, s = torch.empty_like(d["x"]), torch.empty(4, device="cuda")
    y8 = torch.empty((4, 64), dtype=torch.float8_e4m3fn, device="cuda")
    E = cpdr.CpdrError
    bad = [
        (E, "neither y nor y8", lambda: ctx.layernorm_fwd(d["x"], d["w"])),
        (E, "come together", lambda: ctx.layernorm_fwd(d["x"], d["w"], y8=y8)),
        (E, "come together", lambda: ctx.layernorm_fwd(d["x"], d["w"], y=y, scale=s)),
        (E, "overlaps", lambda: ctx.layernorm_fwd(d["x"], d["w"], residual=d["r"], sum_out=d["x"], y=d["x"])),
        (E, "eps", lambda: ctx.layernorm_fwd(d["x"], d["w"], y=y, eps=-1.0)),
        (E, "eps", lambda: ctx.layernorm_fwd(d["x"], d["w"], y=y, eps=float("nan"))),
        (E, "multiple of 8", lambda: ctx.layernorm_fwd(d["x"][:, :12].contiguous(), d["w"][:12], y=y[:, :12].contiguous())),
        (ValueError, "bias must be", lambda: ctx.layernorm_fwd(d["x"], d["w"], bias=d["b"][:8], y=y)),
        (ValueError, "weight must be", lambda: ctx.layernorm_fwd(d["x"], d["w"].bfloat16(), y=y)),
        (E, "workspace", lambda: ctx.layernorm_bwd(d["x"], d["w"], d["dy"],
                                                   workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (E, "overlaps", lambda: ctx.layernorm_bwd(d["x"], d["w"], d["dy"], out=dict(ds=y, dweight=d["w"], dbias=None))),
        (E, "overlaps", lambda: ctx.layernorm_bwd(d["x"], d["w"], d["dy"], out=dict(ds=d["x"], dweight=d["b"], dbias=None))),
    ]
    for kind, what, call in bad:
        with pytest.raises(kind, match=what):
            call()
    wide = torch.empty((1, 16392), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(E, match="16384"):
        ctx.layernorm_fwd(wide, torch.ones(16392, device="cuda"), y=torch.empty_like(wide))
