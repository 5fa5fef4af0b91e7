"""The layer steps at the ends of what their contracts allow: tensors of more
than 2^31 elements, the longest reductions and the most rows and columns that
a form takes, 65535 rows of one state slot, and tensors that begin 16 bytes
past a larger alignment.
"""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol
from test_gpu_glr import close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.empty_cache()


def needs(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_recurrence_past_2_31_elements():
    """Two sequences, the second behind the 2^31st element."""
    needs(60)
    C, last = 2048, 300
    T = (1 << 31) // C + 700
    ctx = cpdr.Context(1, T, 1, 64, 1, dtype="bf16", cu_seqlens=[0, T - last, T])
    x, dy = (torch.zeros(1, T, C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.full((1, T, C), -0.01, device="cuda")
    for at, seed in ((slice(0, 400), 1), (slice(T - last, T), 2)):
        n = at.stop - at.start
        x[0, at], dy[0, at] = randn(seed, n, C).bfloat16(), randn(seed + 9, n, C).bfloat16()
        g[0, at] = torch.nn.functional.logsigmoid(2 + randn(seed + 5, n, C))
    h0, dhT = randn(3, 2, C), randn(4, 2, C)
    y, hT = torch.empty_like(x), torch.empty_like(h0)
    carry = torch.empty(ctx.glr_carry_shape(C), device="cuda")
    ctx.glr_fwd(x, g, y, h0=h0, hT=hT, carry=carry)
    out = ctx.glr_bwd(x, g, carry, dy, dhT=dhT)
    torch.cuda.synchronize()
    ctx.check_device_status()
    pick = slice(5, C, 97)          # the oracle runs some of the channels
    f = ol.glr_forward(x[:, :400, pick], g[:, :400, pick], h0[:1, pick])
    close(y[:, :400, pick], f["y"], f["e_y"], "bf16")
    tail = [t[:, T - last:, pick] for t in (x, g, dy)]
    f = ol.glr_forward(*tail[:2], h0[1:, pick])
    close(y[:, T - last:, pick], f["y"], f["e_y"], "bf16")
    close(hT[1:, pick], f["hT"], f["e_hT"], "fp32")
    b = ol.glr_backward(*tail, h0[1:, pick], dhT[1:, pick])
    close(out["dx"][:, T - last:, pick], b["dx"], b["e_dx"], "bf16")
    close(out["dg"][:, T - last:, pick], b["dg"], b["e_dg"], "fp32")
    close(out["dh0"][1:, pick], b["dh0"], b["e_dh0"], "fp32")


@pytest.mark.parametrize("width", [8, 8200])
def test_norm_past_2_31_elements(width):
    """Rows are independent: the last ones equal a small call's, to the bit."""
    needs(40)
    rows = (1 << 31) // width + 1000
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    x[-500:] = randn(1, 500, width).bfloat16()
    w = 1 + 0.1 * randn(2, width)
    y, y8, scale = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), \
        torch.empty(rows, device="cuda")
    ctx.rmsnorm_fwd(x, w, y=y, y8=y8, scale=scale)
    s = x[-500:].clone()
    a, a8, sc = torch.empty_like(s), torch.empty(s.shape, dtype=torch.float8_e4m3fn, device="cuda"), \
        torch.empty(500, device="cuda")
    ctx.rmsnorm_fwd(s, w, y=a, y8=a8, scale=sc)
    assert torch.equal(y[-500:], a) and torch.equal(y8[-500:].view(torch.uint8), a8.view(torch.uint8))
    assert torch.equal(scale[-500:], sc) and (y[:1000] == 0).all()
    del y8
    out = ctx.rmsnorm_bwd(x, w, y)
    ref = ctx.rmsnorm_bwd(s, w, a)
    assert torch.equal(out["ds"][-500:], ref["ds"])


def test_recurrence_step_with_one_slot_for_65535_rows():
    """Its rows are one sequence: token by token, as the scan runs them."""
    n, C = 65535, 16
    x, g = randn(5, n, C).bfloat16(), torch.nn.functional.logsigmoid(2 + randn(6, n, C))
    state = randn(7, 3, C)
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    y, was = torch.empty_like(x), state.clone()
    ctx.glr_step(x, g, state, y, slots=torch.full((n,), 1, dtype=torch.int32, device="cuda"))
    f = ol.glr_forward(x[None], g[None], was[1:2])
    close(y, f["y"][0], f["e_y"][0], "bf16")
    close(state[1:2], f["hT"], f["e_hT"], "fp32")
    assert torch.equal(state[::2], was[::2])


def product(x, w, mag=False):
    """x w^T in 64 bits on the GPU."""
    x, w = x.double(), w.double()
    return x.abs() @ w.abs().t() if mag else x @ w.t()


@pytest.mark.parametrize("M,K,N", [(1 << 20, 8, 8), ((1 << 20) + 1, 8, 8), (128 * 65535, 8, 8), (128 * 65535 + 1, 8, 136),
                                   (1, 8, 1 << 23), (5, 16, (1 << 23) - 8), (1, 1 << 23, 8), (200, 1 << 20, 72)])
def test_products_at_the_ends_of_their_forms(M, K, N):
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    x, w = randn(8, M, K).bfloat16(), (randn(9, N, K) / K ** 0.5).bfloat16()
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ctx.linear_fwd(x, w, y)
    out = ctx.linear_bwd(x, w, y, out=dict(dx=torch.empty_like(x)))
    torch.cuda.synchronize()
    ctx.check_device_status()
    half = ol.HALF_STEP["bf16"]
    for got, a, b in ((y, x, w), (out["dx"], y, w.t())):
        ref, err = product(a, b), ol._sum_error(a.shape[1]) * product(a, b, True)
        assert ((got.double() - ref).abs() <= err + half * (ref.abs() + err) + 1e-37).all()


def shifted(t):
    """The same values 16 bytes past the allocation's start."""
    skip = 16 // t.element_size()
    flat = torch.empty(t.numel() + skip, dtype=t.dtype, device=t.device)
    out = flat[skip:].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 32 == 16
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tensors_that_begin_16_bytes_on(dtype):
    T, C = 333, 200
    ctx = cpdr.Context(1, T, 1, 64, 1, dtype=dtype)
    dt = ctx.torch_dtype
    x, g, h0 = randn(1, 1, T, C).to(dt), -randn(2, 1, T, C).abs(), randn(3, 1, C)
    w, res = 1 + 0.1 * randn(4, C), randn(5, T, C).to(dt)

    def go(f):
        xs, gs, hs, ws, rs = (f(t) for t in (x, g, h0, w, res))
        empty = {k: f(torch.empty_like(t)) for k, t in (("y", x), ("n", x[0]), ("s", x[0]), ("hT", h0))}
        carry = f(torch.empty(ctx.glr_carry_shape(C), device="cuda"))
        y8, sc = f(torch.zeros(T, C, device="cuda").to(torch.float8_e4m3fn)), f(torch.empty(T, device="cuda"))
        ctx.glr_fwd(xs, gs, empty["y"], h0=hs, hT=empty["hT"], carry=carry)
        b = ctx.glr_bwd(xs, gs, carry, empty["y"], dhT=hs,
                        out=dict(dx=f(torch.empty_like(x)), dg=f(torch.empty_like(g)), dh0=f(torch.empty_like(h0))))
        ctx.rmsnorm_fwd(xs[0], ws, residual=rs, sum_out=empty["s"], y=empty["n"], y8=y8, scale=sc)
        n = ctx.rmsnorm_bwd(empty["s"], ws, empty["n"], dsum=rs,
                            out=dict(ds=f(torch.empty_like(res)), dweight=f(torch.empty_like(w))),
                            workspace=f(torch.empty(ctx.rmsnorm_bwd_workspace_bytes(T, C), dtype=torch.uint8, device="cuda")))
        state, ys = f(h0), f(torch.empty_like(x[0, :1]))
        ctx.glr_step(xs[0, :1], gs[0, :1], state, ys)
        outs = [*empty.values(), carry, y8.view(torch.uint8), sc, *b.values(), *n.values(), state, ys]
        if dtype == "bf16":
            m = f((randn(6, 72, C) / 14).bfloat16())
            bias, r2 = f(randn(7, 72)), f(randn(8, T, 72).bfloat16())
            y2, z = f(torch.empty_like(r2)), f(torch.empty_like(r2))
            ctx.linear_fwd(empty["n"], m, y2, bias=bias, activation="gelu", residual=r2, z=z)
            lb = ctx.linear_bwd(empty["n"], m, y2, z=z, activation="gelu",
                                out=dict(dx=f(torch.empty_like(empty["n"])), dw=f(torch.empty_like(m)), dbias=f(torch.empty_like(bias))))
            outs += [y2, z, *lb.values()]
        torch.cuda.synchronize()
        ctx.check_device_status()
        return outs

    for a, b in zip(go(lambda t: t.clone()), go(shifted)):
        assert torch.equal(a, b)
