"""GPU parity of the matrix product with its epilogue (cpdr_linear_fwd, _bwd)
against the fp64 oracle (oracle/layer_steps.py): both kernels, from one row
to several tiles, sizes that end inside a tile, every combination of bias,
activation and residual, e4m3 operands with scales, each gradient alone and
together, in-place residuals, a captured graph and another stream.

Bars: the oracle's error bounds plus half a step of the output's type.
"""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


@pytest.fixture(scope="module")
def ctx(_cuda):
    return cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")


def draw(M, K, N, seed=0, e4m3=False):
    gen = torch.Generator().manual_seed(M * 7 + K * 3 + N + seed)

    def randn(*s):
        return torch.randn(s, generator=gen)

    d = dict(bias=0.3 * randn(N), residual=randn(M, N).bfloat16(), dy=randn(M, N).bfloat16(), z=(1.5 * randn(M, N)).bfloat16())
    if e4m3:
        d.update(x=randn(M, K).to(torch.float8_e4m3fn), w=randn(N, K).to(torch.float8_e4m3fn),
                 x_scale=torch.exp(0.3 * randn(M)), w_scale=torch.exp(0.3 * randn(N)) / K ** 0.5)
    else:
        d.update(x=randn(M, K).bfloat16(), w=(randn(N, K) / K ** 0.5).bfloat16())
    return d


def close(got, ref, err, dtype="bf16"):
    got = got.double().cpu().numpy()
    tol = err + ol.HALF_STEP[dtype] * (np.abs(ref) + err) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), got.size, float(np.nanmax(np.abs(got - ref) / tol)))


def forward(ctx, M, K, N, act=None, bias=True, residual=True, z=False, e4m3=False):
    d = draw(M, K, N, e4m3=e4m3)
    c = {k: v.cuda() for k, v in d.items()}
    scales = {k: c[k] for k in ("x_scale", "w_scale") if k in c}
    # rows behind the last one are there to be left alone
    y = torch.full((M + 3, N), 7.0, device="cuda").bfloat16()
    zt = torch.full((M + 3, N), 5.0, device="cuda").bfloat16()
    ctx.linear_fwd(c["x"], c["w"], y[:M], bias=c["bias"] if bias else None, activation=act,
                   residual=c["residual"] if residual else None, z=zt[:M] if z else None, **scales)
    torch.cuda.synchronize()
    ctx.check_device_status()
    f = ol.linear_forward(d["x"], d["w"], d["bias"] if bias else None, act, d["residual"] if residual else None,
                          **{k: d[k] for k in scales})
    close(y[:M], f["y"], f["e_y"])
    assert (y[M:] == 7).all()
    if z:
        close(zt[:M], f["z"], f["e_z"])
    assert (zt[M:] == 5).all() and (z or (zt == 5).all())


SIZES = [(1, 64, 64), (1, 8, 8), (3, 72, 136), (16, 256, 128), (17, 520, 1032), (33, 136, 264), (64, 2048, 384),
         (65, 64, 1000), (100, 1096, 520), (129, 264, 128), (255, 512, 256), (257, 200, 264), (512, 128, 1024),
         (1000, 328, 520), (2000, 64, 72), (2304, 512, 2560)]


@pytest.mark.parametrize("M,K,N", SIZES)
def test_bf16_sizes(ctx, M, K, N):
    forward(ctx, M, K, N, act="silu", z=True)


@pytest.mark.parametrize("M,K,N", [(1, 16, 8), (5, 144, 264), (16, 2048, 384), (40, 272, 136), (128, 512, 128),
                                   (300, 400, 520), (1500, 1040, 1288), (2304, 512, 2560)])
def test_e4m3_sizes(ctx, M, K, N):
    forward(ctx, M, K, N, act="gelu", e4m3=True, z=True)
    forward(ctx, M, K, N, bias=False, residual=False, e4m3=True)


@pytest.mark.parametrize("M", [9, 2000])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_epilogues(ctx, M, act, bias, residual):
    forward(ctx, M, 192, 1288 if M > 9 else 264, act=act, bias=bias, residual=residual, z=act is not None)


def test_long_reduction_and_many_tiles(ctx):
    """Several passes of the persistent pairs over the stages, both accumulators in turn."""
    forward(ctx, 5000, 1096, 2056, act=None)


# 90 tiles, the last 14 in halves, one of them with 8 columns; and 24 tiles all in halves
@pytest.mark.parametrize("M,K,N", [(2500, 80, 2184), (900, 336, 1288)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_whole_and_halved_tiles(ctx, M, K, N, residual, e4m3):
    forward(ctx, M, K, N, act="silu", residual=residual, z=True, e4m3=e4m3)
    forward(ctx, M, K, N, act="gelu", residual=residual, e4m3=e4m3)


@pytest.mark.parametrize("M,K,N", [(2500, 2184, 72), (136, 2184, 2504), (900, 1288, 72), (136, 1288, 904)])
def test_gradients_of_whole_and_halved_tiles(ctx, M, K, N):
    backward(ctx, M, K, N, None)


def test_leading_dimensions_are_rows(ctx):
    d = {k: v.cuda() for k, v in draw(24, 64, 72).items()}
    y, y3 = torch.empty(24, 72, device="cuda").bfloat16(), torch.empty(2, 12, 72, device="cuda").bfloat16()
    ctx.linear_fwd(d["x"], d["w"], y)
    ctx.linear_fwd(d["x"].view(2, 12, 64), d["w"], y3)
    assert torch.equal(y, y3.view(24, 72))


def backward(ctx, M, K, N, act):
    d = draw(M, K, N, seed=1)
    c = {k: v.cuda() for k, v in d.items()}
    b = ol.linear_backward(d["x"], d["w"], d["dy"], d["z"], act)
    out = dict(dx=torch.full_like(c["x"], float("nan")), dw=torch.full_like(c["w"], float("nan")),
               dbias=torch.full((N,), float("nan"), device="cuda"))
    z = c["z"] if act else None
    ctx.linear_bwd(c["x"], c["w"], c["dy"], z=z, activation=act, out=out)
    torch.cuda.synchronize()
    ctx.check_device_status()
    close(out["dx"], b["dx"], b["e_dx"])
    close(out["dw"], b["dw"], b["e_dw"])
    close(out["dbias"], b["dbias"], b["e_dbias"], "fp32")
    for k in out:      # each alone: the same bits
        one = {k: torch.empty_like(out[k])}
        ctx.linear_bwd(c["x"], c["w"], c["dy"], z=z, activation=act, out=one)
        assert torch.equal(one[k], out[k]), k


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("M,K,N", [(1, 64, 64), (1, 8, 8), (7, 136, 72), (64, 256, 512), (100, 520, 264), (300, 64, 1032),
                                   (1000, 328, 520), (2100, 264, 520)])
def test_gradients(ctx, M, K, N, act):
    backward(ctx, M, K, N, act)


def test_gradients_over_many_tiles(ctx):
    backward(ctx, 2600, 2056, 1288, "silu")


def test_no_rows(ctx):
    w = torch.randn(72, 64, device="cuda").bfloat16()
    x, y = torch.empty(0, 64, device="cuda").bfloat16(), torch.empty(0, 72, device="cuda").bfloat16()
    ctx.linear_fwd(x, w, y)
    out = dict(dx=x.clone(), dw=torch.full_like(w, 3), dbias=torch.full((72,), 3.0, device="cuda"))
    ctx.linear_bwd(x, w, y, out=out)
    torch.cuda.synchronize()
    assert (out["dw"] == 0).all() and (out["dbias"] == 0).all()


@pytest.mark.parametrize("M", [5, 700])
def test_residual_in_place(ctx, M):
    d = {k: v.cuda() for k, v in draw(M, 256, 520).items()}
    y = torch.empty(M, 520, device="cuda").bfloat16()
    ctx.linear_fwd(d["x"], d["w"], y, bias=d["bias"], activation="gelu", residual=d["residual"])
    stream = d["residual"].clone()
    ctx.linear_fwd(d["x"], d["w"], stream, bias=d["bias"], activation="gelu", residual=stream)
    assert torch.equal(y, stream)


@pytest.mark.parametrize("M", [6, 900])
def test_nan_and_infinity_stay_in_their_rows_and_columns(ctx, M):
    d = {k: v.cuda() for k, v in draw(M, 200, 264).items()}
    d["x"][2, 7] = float("nan")
    d["w"][9, 3] = float("inf")
    y = torch.empty(M, 264, device="cuda").bfloat16()
    ctx.linear_fwd(d["x"], d["w"], y)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[2], want[:, 9] = True, True
    assert torch.equal(bad, want) and torch.isnan(y[2]).all()


def test_same_bits_on_another_stream_and_from_graphs(ctx):
    d = {k: v.cuda() for k, v in draw(600, 264, 520).items()}
    s = {k: v.cuda() for k, v in draw(6, 1096, 520, seed=3).items()}

    def go():
        y, y1 = (torch.empty(m, 520, device="cuda").bfloat16() for m in (600, 6))
        ctx.linear_fwd(d["x"], d["w"], y, bias=d["bias"], activation="silu", residual=d["residual"])
        ctx.linear_fwd(s["x"], s["w"], y1, bias=s["bias"])
        return [y, y1, *ctx.linear_bwd(d["x"], d["w"], d["dy"], z=d["z"], activation="silu").values()]

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
    ctx.check_device_status()
    for a, b, c in zip(ref, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals(ctx):
    x = torch.zeros(4, 64, device="cuda").bfloat16()
    w = torch.zeros(72, 64, device="cuda").bfloat16()
    y = torch.empty(4, 72, device="cuda").bfloat16()

    def refused(call, text, status=cpdr.ERR_INVALID):
        with pytest.raises(cpdr.CpdrError, match=text) as ei:
            call()
        assert ei.value.status == status

    f32 = cpdr.Context(1, 1, 1, 64, 1, dtype="fp32")
    refused(lambda: f32.linear_fwd(x, w, y), "only bf16", cpdr.ERR_UNSUPPORTED)
    refused(lambda: ctx.linear_fwd(x[:, :12].contiguous(), w[:, :12].contiguous(), y), "multiple of 8")
    refused(lambda: ctx.linear_fwd(x, w[:12].contiguous(), y[:, :12].contiguous()), "multiple of 8")
    x8, w8 = x[:, :24].contiguous().to(torch.float8_e4m3fn), w[:, :24].contiguous().to(torch.float8_e4m3fn)
    ones = torch.ones(72, device="cuda")
    refused(lambda: ctx.linear_fwd(x8, w8, y, x_scale=ones[:4], w_scale=ones), "multiple of 16")
    refused(lambda: ctx.linear_fwd(x[:, :72 - 8], w, y, z=y), "overlaps")
    refused(lambda: ctx.linear_bwd(x, w, y, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), "workspace",
            cpdr.ERR_WORKSPACE)
    with pytest.raises(ValueError):
        ctx.linear_fwd(x, w, y, x_scale=ones[:4])
    with pytest.raises(ValueError):
        ctx.linear_bwd(x, w, y, activation="silu")
    with pytest.raises(KeyError):
        ctx.linear_fwd(x, w, y, activation="relu")
