"""GPU parity of the RMS norm (cpdr_rmsnorm_fwd, _bwd) against the fp64
oracle (oracle/layer_steps.py): every group size's widths, odd row counts,
both dtypes, the residual's sum, 8-bit outputs with their scales, in-place
forms, rows of zeros, NaN and infinities, and a captured graph.

Bars: the oracle's error bounds plus half a step of the output's type; e4m3
values within half a step of e4m3 (2^-4 of the value, 2^-10 of the scale
below the normal range) of the unrounded quotient.
"""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def context(dtype):
    return cpdr.Context(1, 1, 1, 64, 1, dtype=dtype)


def draw(rows, width, dtype, seed=0):
    gen = torch.Generator().manual_seed(1000 * width + rows + seed)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16

    def randn(*s):
        return torch.randn(s, generator=gen)

    return dict(x=(randn(rows, width) * torch.exp(randn(rows, 1))).to(dt), r=randn(rows, width).to(dt),
                dy=randn(rows, width).to(dt), dsum=randn(rows, width).to(dt), w=1 + 0.3 * randn(width))


def close(got, ref, err, dtype):
    got = got.double().cpu().numpy()
    tol = err + ol.HALF_STEP[dtype] * (np.abs(ref) + err) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)))


def close_e4m3(y8, scale, ref):
    rs = ol.e4m3_scale(ref)
    s = scale.double().cpu().numpy()
    assert (np.abs(s - rs) <= 2 * ol.ROW * rs).all()
    got = y8.double().cpu().numpy() * s[:, None]
    tol = (2.0 ** -4 + 4 * ol.ROW) * np.abs(ref) + 2.0 ** -10 * s[:, None]
    assert (np.abs(got - ref) <= tol).all()


WIDTHS = [8, 16, 24, 32, 56, 64, 128, 136, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    rows = 37
    d = draw(rows, width, dtype)
    c = {k: v.cuda() for k, v in d.items()}
    ctx = context(dtype)
    for res in (None, "r"):
        f = ol.rmsnorm_forward(d["x"], d["w"], EPS, None if res is None else d[res])
        s, y, y2 = (torch.full_like(c["x"], float("nan")) for _ in range(3))
        y8 = torch.empty((rows, width), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.full((rows,), float("nan"), device="cuda")
        kw = dict(residual=None if res is None else c[res], eps=EPS)
        ctx.rmsnorm_fwd(c["x"], c["w"], sum_out=s, y=y, **kw)
        ctx.rmsnorm_fwd(c["x"], c["w"], y=y2, y8=y8, scale=scale, **kw)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
        close(s, f["s"], 0, dtype)
        # s is rounded to fp32 before it is normalised
        close(y, f["y"], (ol.ROW + 2 * ol.U32) * np.abs(f["y"]), dtype)
        close_e4m3(y8, scale, f["y"])
    for dsum in (None, "dsum"):
        b = ol.rmsnorm_backward(d["x"], d["w"], EPS, d["dy"], None if dsum is None else d[dsum])
        out = ctx.rmsnorm_bwd(c["x"], c["w"], c["dy"], dsum=None if dsum is None else c[dsum], eps=EPS)
        torch.cuda.synchronize()
        close(out["ds"], b["ds"], b["e_ds"], dtype)
        close(out["dweight"], b["dweight"], b["e_dweight"], "fp32")


@pytest.mark.parametrize("rows,width", [(1, 8), (3, 64), (37, 136), (700, 264), (5, 776)])
def test_eps_of_zero(rows, width):
    # groups of threads without a row of their own must not reach dweight
    d = draw(rows, width, "fp32", 11)
    c = {k: v.cuda() for k, v in d.items()}
    ctx = context("fp32")
    f, b = ol.rmsnorm_forward(d["x"], d["w"], 0.0), ol.rmsnorm_backward(d["x"], d["w"], 0.0, d["dy"])
    y = torch.empty_like(c["x"])
    ctx.rmsnorm_fwd(c["x"], c["w"], y=y, eps=0.0)
    out = ctx.rmsnorm_bwd(c["x"], c["w"], c["dy"], eps=0.0)
    torch.cuda.synchronize()
    close(y, f["y"], ol.ROW * np.abs(f["y"]), "fp32")
    close(out["ds"], b["ds"], b["e_ds"], "fp32")
    close(out["dweight"], b["dweight"], b["e_dweight"], "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", [40, 48, 72, 88, 96, 192, 384, 776, 1536, 2560, 5208, 6144, 10000, 12288, 12296, 16376])
def test_widths_between(width, dtype):
    test_widths(width, dtype)


@pytest.mark.parametrize("rows,width", [(1, 64), (2, 2048), (3, 128), (15, 8), (16, 128), (17, 128), (3001, 128),
                                        (2049, 264), (700, 2048)])
def test_rows(rows, width):
    d = draw(rows, width, "bf16", 5)
    c = {k: v.cuda() for k, v in d.items()}
    ctx = context("bf16")
    y = torch.full_like(c["x"], float("nan"))
    ctx.rmsnorm_fwd(c["x"], c["w"], residual=c["r"], y=y, eps=EPS)
    out = ctx.rmsnorm_bwd(c["x"], c["w"], c["dy"], dsum=c["dsum"], eps=EPS)
    torch.cuda.synchronize()
    f = ol.rmsnorm_forward(d["x"], d["w"], EPS, d["r"])
    b = ol.rmsnorm_backward(d["x"], d["w"], EPS, d["dy"], d["dsum"])
    close(y, f["y"], (ol.ROW + 2 * ol.U32) * np.abs(f["y"]), "bf16")
    close(out["ds"], b["ds"], b["e_ds"], "bf16")
    close(out["dweight"], b["dweight"], b["e_dweight"], "fp32")


def test_nothing_is_written_behind_the_last_row():
    ctx = context("bf16")
    x = torch.randn(5, 72, device="cuda").bfloat16()
    w = torch.ones(72, device="cuda")
    y = torch.full((9, 72), 3.0, device="cuda").bfloat16()
    y8 = torch.full((9, 72), 2.0, device="cuda").to(torch.float8_e4m3fn)
    scale = torch.full((9,), 5.0, device="cuda")
    ctx.rmsnorm_fwd(x, w, y=y[:5], y8=y8[:5], scale=scale[:5])
    torch.cuda.synchronize()
    assert (y[5:] == 3).all() and (y8[5:].float() == 2).all() and (scale[5:] == 5).all()


def test_zero_rows_and_zero_rows_of_x():
    ctx = context("fp32")
    w = torch.full((64,), 2.0, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    x[2] = 1.0
    y = torch.empty_like(x)
    y8 = torch.empty((4, 64), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(4, device="cuda")
    ctx.rmsnorm_fwd(x, w, y=y, y8=y8, scale=scale, eps=1e-6)
    out = ctx.rmsnorm_bwd(x, w, torch.ones_like(x))
    torch.cuda.synchronize()
    assert (y[[0, 1, 3]] == 0).all() and (y8.float()[[0, 1, 3]] == 0).all()
    assert (scale[[0, 1, 3]] == 2.0 ** -126).all() and (y8.float()[2] == 448).all()
    assert torch.isfinite(out["ds"]).all() and torch.isfinite(out["dweight"]).all()
    empty = torch.empty(0, 64, device="cuda")
    ctx.rmsnorm_fwd(empty, w, y=torch.empty_like(empty))
    out = ctx.rmsnorm_bwd(empty, w, empty.clone(), out=dict(ds=empty.clone(), dweight=torch.full_like(w, 9)))
    torch.cuda.synchronize()
    assert (out["dweight"] == 0).all()                 # a sum over no rows


def test_nan_and_infinity_stay_in_their_rows():
    ctx = context("bf16")
    x = torch.randn(4, 264, device="cuda").bfloat16()
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    w = torch.ones(264, device="cuda")
    y = torch.empty_like(x)
    y8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(4, device="cuda")
    ctx.rmsnorm_fwd(x, w, y=y, y8=y8, scale=scale)
    torch.cuda.synchronize()
    assert torch.isfinite(y[[0, 3]]).all() and torch.isfinite(y8.float()[[0, 3]]).all()
    assert torch.isnan(y[1]).all() and torch.isnan(scale[[1, 2]]).all()
    assert torch.isnan(y8.float()[[1, 2]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place_forms(dtype):
    d = {k: v.cuda() for k, v in draw(33, 520, dtype, 9).items()}
    ctx = context(dtype)
    s, y = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    ctx.rmsnorm_fwd(d["x"], d["w"], residual=d["r"], sum_out=s, y=y)
    x, r = d["x"].clone(), d["r"].clone()
    ctx.rmsnorm_fwd(x, d["w"], residual=r, sum_out=r, y=x)      # the stream and the branch, both in place
    ref = ctx.rmsnorm_bwd(s, d["w"], d["dy"], dsum=d["dsum"])
    for name in ("dy", "dsum"):
        t = dict(dy=d["dy"].clone(), dsum=d["dsum"].clone())
        out = ctx.rmsnorm_bwd(s, d["w"], t["dy"], dsum=t["dsum"],
                              out=dict(ds=t[name], dweight=torch.empty_like(d["w"])))
        assert torch.equal(out["ds"], ref["ds"]) and torch.equal(out["dweight"], ref["dweight"])
    torch.cuda.synchronize()
    assert torch.equal(r, s) and torch.equal(x, y)


def test_graph_and_stream_give_the_same_bits():
    d = {k: v.cuda() for k, v in draw(500, 1032, "bf16", 11).items()}
    ctx = context("bf16")

    def go():
        s, y = torch.empty_like(d["x"]), torch.empty_like(d["x"])
        ctx.rmsnorm_fwd(d["x"], d["w"], residual=d["r"], sum_out=s, y=y)
        return [s, y, *ctx.rmsnorm_bwd(s, d["w"], d["dy"], dsum=d["dsum"]).values()]

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
    ctx = context("bf16")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    y = torch.empty_like(x)
    y8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")

    def refused(call, text, status=cpdr.ERR_INVALID):
        with pytest.raises(cpdr.CpdrError, match=text) as ei:
            call()
        assert ei.value.status == status

    refused(lambda: ctx.rmsnorm_fwd(x, w), "neither y nor y8")
    refused(lambda: ctx.rmsnorm_fwd(x, w, y8=y8), "y8 and scale")
    refused(lambda: ctx.rmsnorm_fwd(x, w, y=y, sum_out=y), "overlaps")
    refused(lambda: ctx.rmsnorm_fwd(x, w, y=y, eps=-1.0), "eps")
    refused(lambda: ctx.rmsnorm_fwd(x, w, y=y, eps=float("nan")), "eps")
    refused(lambda: ctx.rmsnorm_fwd(x.view(-1)[:240].view(20, 12), w[:12], y=y.view(-1)[:240].view(20, 12)), "multiple of 8")
    wide = torch.zeros(1, 16392, dtype=torch.bfloat16, device="cuda")
    refused(lambda: ctx.rmsnorm_fwd(wide, torch.ones(16392, device="cuda"), y=torch.empty_like(wide)), "at most 16384",
            cpdr.ERR_UNSUPPORTED)
    refused(lambda: ctx.rmsnorm_bwd(x, w, y, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), "workspace",
            cpdr.ERR_WORKSPACE)
    part = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    refused(lambda: ctx.rmsnorm_fwd(part[:4], w, y=part[2:6]), "y overlaps x")
    with pytest.raises(ValueError):
        ctx.rmsnorm_fwd(x, w[:32], y=y)
    with pytest.raises(ValueError):
        ctx.rmsnorm_fwd(x, w, y=y.float())
