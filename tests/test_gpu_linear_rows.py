"""The weight gradient over so many rows that a tile's sum outlasts the usual
limit of a wait (4e9 cycles): the sum is still whole, and no wait gives up."""
import pytest
import torch

from context_merge_gb300 import cpdr

pytestmark = pytest.mark.gpu


def test_a_sum_that_outlasts_the_usual_wait(cpdr_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    rows = 1_200_000_013
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(rows, 8, dtype=torch.bfloat16, device="cuda")
    at = [0, 63, 64, rows // 2, rows - 14, rows - 1]
    for i, r in enumerate(at):
        x[r] = torch.arange(8, device="cuda").bfloat16() + 2 ** i
        dy[r] = torch.arange(8, device="cuda").bfloat16() - 3
    ctx = cpdr.Context(1, 1, 1, 64, 1, dtype="bf16")
    out = ctx.linear_bwd(x, torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda"), dy,
                         out=dict(dw=torch.empty(8, 8, dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    ctx.check_device_status()
    # the other rows of x are zero: sums of six products of small whole numbers, exact in fp32
    ref = dy[at].double().t() @ x[at].double()
    assert torch.equal(out["dw"], ref.bfloat16())
