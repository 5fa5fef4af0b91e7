"""GPU parity of the embedding (cpdr_embed_fwd, _bwd): the lookup to the bit
against a gather, its gradient against the fp64 oracle (oracle/model_steps.py)
within the roundings of each token's sum plus half a step of the output's type;
tokens in every share of the batch, padding, odd vocabularies and widths."""
import numpy as np
import pytest
import torch

from context_merge_gb300 import cpdr
from oracle import layer_steps as ol
from oracle import model_steps as om

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def context(dtype):
    return cpdr.Context(1, 1, 1, 64, 1, dtype=dtype)


def ids(kind, n, vocab, seed=0):
    """Tokens: uniform, one in every place, text-like (many of few), each at most once, some outside the table."""
    gen = torch.Generator().manual_seed(17 * n + vocab + seed)
    if kind == "one":
        t = torch.full((n,), vocab - 1)
    elif kind == "text":
        t = (vocab ** torch.rand(n, generator=gen, dtype=torch.float64)).long() - 1
    elif kind == "once":
        t = torch.randperm(vocab, generator=gen)[:n]
    else:
        t = torch.randint(0, vocab, (n,), generator=gen)
    if kind == "pads":
        t[torch.rand(n, generator=gen) < 0.3] = -1
        t[n // 2] = vocab
        t[n // 3] = -(2 ** 31)
        t[-1] = 2 ** 31 - 1
    return t.to(torch.int32)


def lookup(tokens, table, scale):
    live = (tokens >= 0) & (tokens < len(table))
    y = (table[torch.where(live, tokens, 0).long()].float() * scale).to(table.dtype)
    return torch.where(live[..., None], y, torch.zeros_like(y))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,vocab,width", [(1, 1, 8), (1, 5, 16), (3, 7, 24), (64, 100, 64), (257, 1000, 136),
                                           (1000, 31, 1360), (33, 50, 2056), (7, 9, 5208), (3, 4, 20000)])
def test_lookup(n, vocab, width, dtype):
    gen = torch.Generator().manual_seed(n + width)
    table = torch.randn((vocab, width), generator=gen).to(DT[dtype])
    ctx = context(dtype)
    for kind, scale in (("uniform", 1.0), ("pads", 1.7)):
        t = ids(kind, n, vocab)
        y = torch.full((n, width), float("nan"), device="cuda").to(DT[dtype])
        ctx.embed_fwd(t.cuda(), table.cuda(), y, scale=scale)
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), lookup(t, table, np.float32(scale).item()))


def check_gradient(tokens, vocab, width, dtype, scale=1.0, seed=0):
    n = tokens.numel()
    gen = torch.Generator().manual_seed(seed + n)
    dy = torch.randn((n, width), generator=gen).to(DT[dtype])
    ctx = context(dtype)
    out = torch.full((vocab, width), float("nan"), device="cuda").to(DT[dtype])
    got = ctx.embed_bwd(tokens.cuda(), dy.cuda(), out, scale=scale)
    torch.cuda.synchronize()
    assert got is out
    r = om.embed_backward(tokens, dy, vocab, np.float32(scale).item())
    got = got.double().cpu().numpy()
    tol = r["e_dtable"] + ol.HALF_STEP[dtype] * (np.abs(r["dtable"]) + r["e_dtable"])
    bad = ~(np.abs(got - r["dtable"]) <= tol)
    assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["uniform", "one", "text", "pads"])
@pytest.mark.parametrize("n,vocab,width", [(1, 1, 8), (3, 1000, 16), (63, 10, 64), (64, 10, 72), (65, 10, 64), (200, 3, 136),
                                           (2048, 255, 24), (2049, 256, 8), (4500, 257, 40), (700, 70000, 8)])
def test_gradient(n, vocab, width, kind, dtype):
    check_gradient(ids(kind, n, vocab), vocab, width, dtype, scale=1.0 if kind == "one" else 2.5)


@pytest.mark.parametrize("width", [264, 1360, 2048, 2056, 4104])
def test_gradient_widths(width):
    for dtype in ("bf16", "fp32"):
        check_gradient(ids("text", 300, 50), 50, width, dtype)


def test_gradient_of_tokens_that_occur_once_is_exact():
    """Each row alone: dtable is dy's row, to the bit, and zeros elsewhere."""
    t = ids("once", 900, 5000)
    dy = torch.randn((900, 72), generator=torch.Generator().manual_seed(1)).bfloat16()
    out = torch.full((5000, 72), 9.0, device="cuda").bfloat16()
    context("bf16").embed_bwd(t.cuda(), dy.cuda(), out)
    want = torch.zeros((5000, 72)).bfloat16()
    want[t.long()] = dy
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("kind", ["uniform", "one", "text", "pads"])
def test_many_tokens(kind):
    """More tokens than one block's share of every step: in 64 bits on the GPU."""
    n, V, D = 150001, 40001, 64
    t = ids(kind, n, V, seed=3).cuda()
    dy = torch.randn((n, D), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    out = torch.empty((V, D), device="cuda")
    ctx = context("fp32")
    ctx.embed_bwd(t, dy, out, scale=0.5)
    live = (t >= 0) & (t < V)
    at = torch.where(live, t, V).long()

    def sums(x):
        return torch.zeros((V + 1, D), device="cuda", dtype=torch.float64).index_add_(0, at, x.double())[:V]

    ref, mag = 0.5 * sums(dy), 0.5 * sums(dy.abs())
    count = torch.bincount(at, minlength=V + 1)[:V, None]
    # roundings along a path of the sum: at most one per row, and the scale's
    assert ((out.double() - ref).abs() <= (count + 2) * ol.U32 * mag + ol.U32 * ref.abs()).all()
    again = torch.empty_like(out)
    ctx.embed_bwd(t, dy, again, scale=0.5)
    assert torch.equal(out, again)


def test_no_tokens_and_only_padding():
    ctx = context("bf16")
    table = torch.randn((5, 64), device="cuda").bfloat16()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    ctx.embed_fwd(none, table, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    for t in (none, torch.full((130,), -1, dtype=torch.int32, device="cuda")):
        out = torch.full_like(table, 3.0)
        ctx.embed_bwd(t, torch.full((t.numel(), 64), float("nan"), device="cuda").bfloat16(), out)
        torch.cuda.synchronize()
        assert (out == 0).all()


def test_nan_stays_in_its_token():
    t = torch.tensor([3, 1, 3, 0, -1], dtype=torch.int32, device="cuda")
    dy = torch.ones((5, 8), device="cuda")
    dy[0, 2] = dy[4, 1] = float("nan")
    out = torch.empty((5, 8), device="cuda")
    context("fp32").embed_bwd(t, dy, out)
    want = torch.tensor([1.0, 1, 0, 2, 0], device="cuda")[:, None].repeat(1, 8)
    want[3, 2] = float("nan")
    assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0))


def test_batched_tokens():
    """Tokens of any shape: [B, T] with y and dy [B, T, D]."""
    t = ids("pads", 60, 11).reshape(3, 20).cuda()
    table = torch.randn((11, 32), device="cuda")
    y = torch.empty((3, 20, 32), device="cuda")
    ctx = context("fp32")
    ctx.embed_fwd(t, table, y)
    a, b = torch.empty_like(table), torch.empty_like(table)
    ctx.embed_bwd(t, y, a)
    ctx.embed_bwd(t.view(-1), y.view(60, 32), b)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), lookup(t.cpu(), table.cpu(), 1.0)) and torch.equal(a, b)


def test_offsets_past_2_31_elements():
    """A table of 2.2e9 elements, whose last rows occur."""
    V, D = 2 ** 31 // 8192 + 300, 8192
    table = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    table[-1], table[0] = 2.0, 3.0
    t = torch.tensor([V - 1, 0, V - 2, V - 1], dtype=torch.int32, device="cuda")
    y = torch.empty((4, D), dtype=torch.bfloat16, device="cuda")
    ctx = context("bf16")
    ctx.embed_fwd(t, table, y)
    assert [float(r.min()) for r in y] == [2.0, 3.0, 0.0, 2.0] == [float(r.max()) for r in y]
    ctx.embed_bwd(t, y, table)
    torch.cuda.synchronize()
    assert (table[-1] == 4.0).all() and (table[0] == 3.0).all() and (table[1:-1] == 0).all()


def test_refusals():
    ctx = context("bf16")
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((3, 16), dtype=torch.bfloat16, device="cuda")
    E = cpdr.CpdrError
    bad = [
        (E, "finite", lambda: ctx.embed_fwd(t, table, y, scale=float("inf"))),
        (E, "finite", lambda: ctx.embed_bwd(t, y, table, scale=float("nan"))),
        (E, "multiple of 8", lambda: ctx.embed_fwd(t, table[:, :12].contiguous(), y[:, :12].contiguous())),
        (E, "vocab", lambda: ctx.embed_fwd(t, table[:0], y)),
        (E, "overlaps", lambda: ctx.embed_fwd(t, table, table[:3])),
        (E, "overlaps", lambda: ctx.embed_bwd(t, table[:3], table)),
        (E, "workspace", lambda: ctx.embed_bwd(t, y, table, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
        (ValueError, "tokens must be", lambda: ctx.embed_fwd(t.long(), table, y)),
        (ValueError, "y must be", lambda: ctx.embed_fwd(t, table, y[:2])),
        (ValueError, "table must be", lambda: ctx.embed_fwd(t, table.float(), y)),
        (ValueError, "dy must be", lambda: ctx.embed_bwd(t, y.float(), table)),
    ]
    for kind, what, call in bad:
        with pytest.raises(kind, match=what):
            call()
