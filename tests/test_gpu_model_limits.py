"""The model steps at the ends of their contracts: more than 2^31 elements, long
batches, rows and slots that nothing names, no rows at all."""
import pytest
import torch

from context_merge_gb300 import cpdr

pytestmark = pytest.mark.gpu

BIG = 2 ** 31
bf = dict(dtype=torch.bfloat16, device="cuda")


@pytest.fixture(scope="module")
def ctx(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    return cpdr.Context(1, 1, 2, 64, 1, dtype="bf16", conv_width=4)


def test_layernorm_past_2_31_elements(ctx):
    """A row's results do not depend on the rows before it: the last ones equal those of a call of their own."""
    D, last = 2048, 9
    rows = BIG // D + last
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, dy = torch.zeros((rows, D), **bf), torch.zeros((rows, D), **bf)
    x[-last:], dy[-last:] = (torch.randn((last, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    w, b = (torch.randn(D, generator=gen, device="cuda") for _ in range(2))
    y, y8, sc = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    ctx.layernorm_fwd(x, w, bias=b, y=y, y8=y8, scale=sc)
    small = torch.empty((last, D), **bf)
    ctx.layernorm_fwd(x[-last:].clone(), w, bias=b, y=small)
    assert torch.equal(y[-last:], small) and torch.equal(y[0], b.bfloat16())
    assert (y8[-last:].float() * sc[-last:, None] - small.float()).abs().max() <= 0.08 * small.float().abs().max()
    one = ctx.layernorm_bwd(x[-last:].clone(), w, dy[-last:].clone())
    many = ctx.layernorm_bwd(x, w, dy, out=dict(ds=y, dweight=torch.empty_like(w), dbias=torch.empty_like(w)))
    torch.cuda.synchronize()
    assert torch.equal(many["ds"][-last:], one["ds"]) and (many["ds"][0] == 0).all()


def test_embedding_past_2_31_elements(ctx):
    """A batch of a million rows: every row of y is its token's, and a table's gradient of ones counts its tokens."""
    D, V = 2048, 1000
    n = BIG // D + 77
    gen = torch.Generator(device="cuda").manual_seed(2)
    tok = torch.randint(-1, V, (n,), generator=gen, device="cuda").to(torch.int32)
    table = torch.arange(V, device="cuda").bfloat16()[:, None].repeat(1, D)
    y = torch.empty((n, D), **bf)
    ctx.embed_fwd(tok, table, y)
    want = torch.where(tok >= 0, tok, 0).bfloat16()
    assert torch.equal(y[:, 0], want) and torch.equal(y[:, -1], want) and torch.equal(y[-1], want[-1].expand(D))
    y.fill_(1.0)
    ctx.embed_bwd(tok, y, table)
    torch.cuda.synchronize()
    count = torch.bincount(tok.long() + 1, minlength=V + 1)[1:].bfloat16()
    assert torch.equal(table, count[:, None].expand(V, D))


def test_conv_pool_past_2_31_elements(ctx):
    C = 8192
    S = BIG // (3 * C) + 50
    gen = torch.Generator(device="cuda").manual_seed(3)
    pool = torch.zeros((S, 3, C), **bf)
    slots = [S - 1, 0, BIG // (3 * C)]
    state = torch.randn((3, 3, C), generator=gen, device="cuda").bfloat16()
    pool[slots] = state
    x, w = torch.randn((3, C), generator=gen, device="cuda").bfloat16(), torch.randn((C, 4), generator=gen, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    ctx.conv1d_step(x, w, None, pool, y, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    ctx.conv1d_step(x, w, None, state, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(pool[slots], state) and (pool[1] == 0).all() and (pool[S - 2] == 0).all()


@pytest.mark.parametrize("n", [4095, 4096, 4097, 8193, 524288, 524289])
def test_batches_around_the_sorts_tiles(ctx, n):
    """Batches that fill the sort's tiles to the last pair and one more."""
    V, D = 3000, 8
    tok = torch.randint(0, V, (n,), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").to(torch.int32)
    out = torch.empty((V, D), **bf)
    ctx.embed_bwd(tok, torch.ones((n, D), **bf), out)
    torch.cuda.synchronize()
    assert torch.equal(out, torch.bincount(tok.long(), minlength=V).bfloat16()[:, None].expand(V, D))


@pytest.mark.parametrize("run", [17, 47, 48, 49, 63, 64, 65, 80, 81, 129, 160, 161, 192, 193, 300, 8192, 8193])
def test_runs_around_the_sums_segments(ctx, run):
    """One token in `run` places among others, from every place of a segment on: whole sums, and those in parts."""
    for before in (0, 1, 31, 32, 33):
        n, D = before + run + 40, 40
        tok = torch.full((n,), 7, dtype=torch.int32)
        tok[:before] = torch.arange(before) % 7
        tok[before + run:] = 8 + torch.arange(40) // 3
        perm = torch.randperm(n, generator=torch.Generator().manual_seed(run + before))
        dy = torch.randint(-4, 5, (n, D), generator=torch.Generator().manual_seed(before)).float()
        want = torch.zeros((30, D)).index_add_(0, tok.long(), dy)
        out = torch.empty((30, D), device="cuda")
        f32 = cpdr.Context(1, 1, 1, 64, 1, dtype="fp32")
        f32.embed_bwd(tok[perm].cuda(), dy[perm].cuda(), out)
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)      # whole numbers: no rounding


def test_no_rows(ctx):
    e = torch.empty
    ctx.layernorm_fwd(e((0, 64), **bf), torch.ones(64, device="cuda"), y=e((0, 64), **bf))
    state = torch.ones((3, 2, 64, 64), device="cuda")
    ctx.delta_step(*(e((0, 2, 64), **bf) for _ in range(3)), e((0, 2), **bf), e((0, 2), device="cuda"), state, e((0, 2, 64), **bf))
    win = torch.ones((3, 3, 16), **bf)
    ctx.conv1d_step(e((0, 16), **bf), torch.ones((16, 4), device="cuda"), None, win, e((0, 16), **bf))
    torch.cuda.synchronize()
    assert (state == 1).all() and (win == 1).all()


@pytest.mark.parametrize("run", [120, 128, 129, 159, 160, 161, 162, 300, 70000])
def test_runs_around_the_sums_segments_of_large_batches(ctx, run):
    """The same in a batch of so many segments that runs may go on further: 1400 blocks of them."""
    n, D, V = 45000, 2048, 400
    if run > n:
        n = run + 5000
    gen = torch.Generator(device="cuda").manual_seed(run)
    tok = torch.randint(8, V, (n,), generator=gen, device="cuda").to(torch.int32)
    tok[torch.randperm(n, generator=gen, device="cuda")[:run]] = 7
    tok[tok == 8] = 7 if run > 1000 else 9
    dy = torch.randint(-4, 5, (n, D), generator=gen, device="cuda").float()
    f32 = cpdr.Context(1, 1, 1, 64, 1, dtype="fp32")
    out = torch.empty((V, D), device="cuda")
    f32.embed_bwd(tok, dy, out)
    torch.cuda.synchronize()
    # whole numbers: no rounding, in any order
    assert torch.equal(out, torch.zeros((V, D), device="cuda").index_add_(0, tok, dy))


@pytest.mark.parametrize("n", [3000, 5000])
@pytest.mark.parametrize("V", [1023, 1024, 2 ** 20 - 1, 2 ** 20, 2 ** 21 + 3, 2 ** 30])
def test_vocabularies_of_one_to_four_sorting_passes(ctx, V, n):
    """Tokens at both ends of the vocabulary and between, padding on either side of it; everything else is zero."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    some = torch.cat([torch.randint(0, V, (40,), generator=gen, device="cuda"), torch.tensor([0, V - 1, -1, V], device="cuda")])
    tok = some[torch.randint(0, 44, (n,), generator=gen, device="cuda")].to(torch.int32)
    dy = torch.randint(0, 2, (n, 8), generator=gen, device="cuda").bfloat16()
    out = torch.full((V, 8), 3.0, **bf)
    ctx.embed_bwd(tok, dy, out)
    torch.cuda.synchronize()
    live = (tok >= 0) & (tok < V)
    ids, at = torch.unique(tok[live].long(), return_inverse=True)
    want = torch.zeros((len(ids), 8), device="cuda").index_add_(0, at, dy[live].float())
    assert torch.equal(out[ids], want.bfloat16())
    out[ids] = 0
    assert not out.view(torch.int64).any()
