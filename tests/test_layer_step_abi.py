"""Refusals of the layer steps' entry points, decided on the host before any
launch (no GPU): null and misaligned pointers, sizes, overlapping tensors.
A host-only context refuses every launch; the Python binding refuses wrong
shapes, dtypes and devices."""
import ctypes

import pytest
import torch

from context_merge_gb300 import cpdr


def make(**kw):
    base = dict(B=1, T=64, H=1, d=64, R=1, dtype="bf16", host_only=True)
    base.update(kw)
    return cpdr.Context(**base)


def P(x):
    return ctypes.c_void_p(x)


def test_host_only_context_rejects_launches(cpdr_lib):
    c = make()
    calls = [
        lambda: cpdr_lib.cpdr_glr_fwd(c._h, P(16), P(32), None, 8, P(48), None, None, None),
        lambda: cpdr_lib.cpdr_glr_bwd(c._h, P(16), P(32), P(48), P(64), None, 8, P(80), P(96), None, None),
        lambda: cpdr_lib.cpdr_glr_step(c._h, P(16), P(32), P(48), P(48), None, 1, 1, 8, P(64), None),
        lambda: cpdr_lib.cpdr_rmsnorm_fwd(c._h, 1, 8, P(16), None, P(32), 1e-6, None, P(48), None, None, None),
        lambda: cpdr_lib.cpdr_rmsnorm_bwd(c._h, 1, 8, P(16), P(32), 1e-6, P(48), None, P(64), P(80), P(96), 1 << 20, None),
        lambda: cpdr_lib.cpdr_linear_fwd(c._h, 1, 8, 8, P(16), P(32), None, None, None, 0, None, None, P(48), None),
        lambda: cpdr_lib.cpdr_linear_bwd(c._h, 1, 8, 8, P(16), P(32), None, P(48), 0, P(64), None, None, None, 0, None),
    ]
    for call in calls:
        assert call() == cpdr.ERR_INVALID
        assert b"HOST_ONLY" in cpdr_lib.cpdr_last_error()


@pytest.mark.parametrize("lengths,groups", [([64], 4), ([1, 15, 16, 17, 0, 15], 6), ([63, 1], 5)])
def test_carry_holds_the_state_before_every_16th_token(cpdr_lib, lengths, groups):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    c = make(T=cu[-1], cu_seqlens=cu)
    assert c.glr_carry_shape(24) == (groups, 24)
    n = ctypes.c_size_t()
    for bad in (0, -8, 12):
        assert cpdr_lib.cpdr_glr_carry_bytes(c._h, bad, ctypes.byref(n)) == cpdr.ERR_INVALID
    assert cpdr_lib.cpdr_glr_carry_bytes(c._h, 8, None) == cpdr.ERR_INVALID


def test_binding_refuses_tensors_that_are_not_on_the_gpu(cpdr_lib):
    c = make()
    x = torch.zeros(1, 64, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be on"):
        c.glr_fwd(x, torch.zeros(1, 64, 8), torch.zeros_like(x))
    with pytest.raises(ValueError, match="must be on"):
        c.rmsnorm_fwd(x, torch.ones(8), y=torch.zeros_like(x))
    with pytest.raises(ValueError, match="must be on"):
        c.glr_step(x[0], torch.zeros(64, 8), torch.zeros(64, 8), x[0].clone())


def test_binding_refuses_wrong_shapes_and_dtypes(cpdr_lib):
    c = make()
    x = torch.zeros(1, 64, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be"):
        c.glr_fwd(x[:, :5], torch.zeros(1, 5, 8), x)
    with pytest.raises(ValueError, match="contiguous"):
        c.rmsnorm_fwd(x.float(), torch.ones(8), y=x)
    with pytest.raises(ValueError, match="state"):
        c.glr_step(x, x, torch.zeros(8), x)
