"""Every form that the matrix product's dispatch can pick, against the fp64
oracle: tiles of 16 to 128 rows of x, the reduction split over 1 to 8 CTAs
(splits that do not divide a tile's columns leave owners short or empty), and
the form for many rows; in bf16, e4m3 and as the input gradient.

The sizes are the cheapest of a random search for each form that end inside a
tile of rows, a tile of 128 columns and a block of the reduction; the plan
(Context.linear_plan) says that they run in it.
"""
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol
from test_gpu_linear import close, draw, forward

# (rows of x in a tile, split) -> rows, K, N; tiles of 0 rows: the form for many rows
BF16 = {
    (0, 1): (2456, 8, 392), (16, 1): (9, 8, 136), (16, 2): (9, 72, 136), (16, 3): (9, 136, 136),
    (16, 4): (9, 392, 136), (16, 5): (11, 608, 136), (16, 6): (9, 1032, 136), (16, 7): (9, 1328, 144),
    (16, 8): (10, 1968, 136), (32, 1): (2435, 8, 136), (32, 2): (761, 136, 136), (32, 3): (1246, 144, 136),
    (32, 4): (458, 1416, 136), (32, 5): (434, 1552, 136), (32, 6): (319, 3056, 136), (32, 7): (311, 3128, 168),
    (32, 8): (259, 5448, 144), (64, 2): (1546, 416, 136), (64, 3): (1257, 1056, 160), (64, 4): (807, 2984, 136),
    (64, 5): (824, 3408, 136), (64, 6): (632, 6344, 136), (64, 7): (232, 6648, 528), (64, 8): (509, 12136, 136),
    (128, 2): (2439, 80, 136), (128, 3): (2569, 1488, 136), (128, 4): (1809, 5608, 144),
    (128, 5): (1539, 5520, 136), (128, 6): (1383, 12120, 176), (128, 7): (1113, 11576, 136)
}
E4M3 = {
    (0, 1): (2451, 16, 392), (16, 1): (9, 16, 136), (16, 2): (9, 144, 136), (16, 3): (10, 272, 136),
    (16, 4): (9, 800, 136), (16, 5): (9, 1168, 144), (16, 6): (9, 2192, 144), (16, 7): (11, 2672, 136),
    (16, 8): (9, 3952, 136), (32, 1): (2435, 16, 136), (32, 2): (1246, 144, 136), (32, 3): (1231, 272, 136),
    (32, 4): (403, 2960, 152), (32, 5): (437, 3088, 144), (32, 6): (350, 5808, 136), (32, 7): (305, 6224, 144),
    (32, 8): (257, 10960, 136), (64, 2): (1618, 832, 144), (64, 3): (1221, 2224, 136), (64, 4): (833, 5456, 144),
    (64, 5): (524, 5664, 264), (64, 6): (388, 11952, 264), (64, 7): (107, 12368, 1272),
    (128, 2): (2494, 144, 136), (128, 3): (2460, 2960, 160), (128, 4): (1893, 11440, 136),
    (128, 5): (1501, 11200, 144)
}


@pytest.fixture(scope="module")
def ctx(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    return cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")


@pytest.mark.parametrize("e4m3,sizes", [(False, BF16), (True, E4M3)])
def test_the_sizes_run_in_their_forms(cpdr_lib, e4m3, sizes):
    c = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16", host_only=True)
    assert {k: c.linear_plan(*v, e4m3=e4m3) for k, v in sizes.items()} == {k: k for k in sizes}
    assert {q for q, _ in sizes} == {0, 16, 32, 64, 128} and {s for _, s in sizes} == set(range(1, 9))


def test_plan_refusals(cpdr_lib):
    c = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16", host_only=True)
    for bad in ((0, 64, 64), (-1, 64, 64), (4, 12, 64), (4, 64, 0)):
        with pytest.raises(cpdr.CpdrError):
            c.linear_plan(*bad)
    with pytest.raises(cpdr.CpdrError):
        c.linear_plan(4, 24, 64, e4m3=True)
    with pytest.raises(cpdr.CpdrError):
        cpdr.Context(1, 1, 1, 64, 1, dtype="fp32", host_only=True).linear_plan(4, 64, 64)
    assert cpdr_lib.cpdr_plan_linear(c._h, 4, 64, 64, 0, None) == cpdr.ERR_INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("form", sorted(BF16))
def test_forward(ctx, form):
    M, K, N = BF16[form]
    assert ctx.linear_plan(M, K, N) == form
    forward(ctx, M, K, N, act="silu", z=True)


@pytest.mark.gpu
@pytest.mark.parametrize("form", sorted(E4M3))
def test_e4m3(ctx, form):
    M, K, N = E4M3[form]
    assert ctx.linear_plan(M, K, N, e4m3=True) == form
    forward(ctx, M, K, N, act="gelu", e4m3=True)


@pytest.mark.gpu
@pytest.mark.parametrize("form", sorted(BF16))
def test_input_gradient(ctx, form):
    """dx = dy w: a product over N with w read along K."""
    M, N, K = BF16[form]
    assert ctx.linear_plan(M, N, K) == form
    d = draw(M, K, N, seed=2)
    # rows behind the last one are there to be left alone
    dx = torch.full((M + 3, K), 7.0, device="cuda").bfloat16()
    ctx.linear_bwd(d["x"].cuda(), d["w"].cuda(), d["dy"].cuda(), out=dict(dx=dx[:M]))
    torch.cuda.synchronize()
    ctx.check_device_status()
    dy, w = d["dy"].double(), d["w"].double()
    close(dx[:M], (dy @ w).numpy(), ol._sum_error(N) * (dy.abs() @ w.abs()).numpy())
    assert (dx[M:] == 7).all()
