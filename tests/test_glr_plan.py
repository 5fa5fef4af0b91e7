"""The recurrence's cluster size: chosen for as many CTAs of an SM as really
fit there, so that the clusters that it counts on run at once."""
import ctypes

import pytest
import torch

from context_merge_gb300 import cpdr


def plan(T, seqs, channels, dtype, backward=False, **kw):
    cu = [i * T // seqs for i in range(seqs)] + [T]
    c = cpdr.Context(1, T, 1, 64, 1, dtype=dtype, cu_seqlens=cu, **kw)
    return c.glr_plan(channels, backward)


# 64 items of 32768 or 65536 tokens: clusters of 8 run 36 at a time, so in two
# rounds, clusters of 4 all at once; 40 and 120 items as the same estimate gives.
@pytest.mark.parametrize("T,seqs,channels,cluster", [(65536, 1, 4096, 4), (65536, 2, 2048, 4), (32768, 1, 2048, 8),
                                                     (32768 * 3, 3, 2560, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_clusters_that_run_at_once(cpdr_lib, T, seqs, channels, cluster, dtype):
    p = plan(T, seqs, channels, dtype, host_only=True)
    assert p == dict(cluster=cluster, per_sm=2, resident=0)


def test_refusals(cpdr_lib):
    c = cpdr.Context(1, 64, 1, 64, 1, dtype="bf16", host_only=True)
    out = (ctypes.c_int32 * 3)()
    for bad in (0, -8, 12):
        assert cpdr_lib.cpdr_plan_glr(c._h, bad, 0, out) == cpdr.ERR_INVALID
    assert cpdr_lib.cpdr_plan_glr(c._h, 8, 0, None) == cpdr.ERR_INVALID
    assert cpdr_lib.cpdr_plan_glr(None, 8, 0, out) == cpdr.ERR_INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("layout", ["contiguous", "zigzag"])
def test_counted_on_is_what_the_device_holds(cpdr_lib, dtype, backward, layout):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    c = cpdr.Context(1, 4096, 1, 64, 2, dtype=dtype, layout=layout)
    p = c.glr_plan(1024, backward)
    assert p["per_sm"] == p["resident"], p
