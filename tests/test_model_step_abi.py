"""Refusals of the model steps' entry points (layer norm, embedding, the mixers'
token steps), decided on the host before any launch (no GPU)."""
import ctypes

import pytest
import torch

from context_merge_gb300 import cpdr


def make(**kw):
    base = dict(B=1, T=64, H=2, d=64, R=1, dtype="bf16", host_only=True, conv_width=4)
    base.update(kw)
    return cpdr.Context(**base)


def P(x):
    return ctypes.c_void_p(x)


def test_host_only_context_rejects_launches(cpdr_lib):
    c = make()
    L = cpdr_lib
    calls = [
        lambda: L.cpdr_layernorm_fwd(c._h, 1, 8, P(16), None, P(32), None, 1e-5, None, P(48), None, None, None),
        lambda: L.cpdr_layernorm_bwd(c._h, 1, 8, P(16), P(32), 1e-5, P(48), None, P(64), P(80), None, P(96), 1 << 20, None),
        lambda: L.cpdr_embed_fwd(c._h, P(16), 1, P(32), 4, 8, 1.0, P(48), None),
        lambda: L.cpdr_embed_bwd(c._h, P(16), 1, 4, 8, 1.0, P(48), P(64), P(80), 1 << 20, None),
        lambda: L.cpdr_delta_step(c._h, P(16), P(32), P(48), P(64), P(80), P(96), P(96), None, 1, 1, P(112), None),
        lambda: L.cpdr_conv1d_step(c._h, P(16), P(32), None, P(48), P(48), None, 1, 1, 8, 1, P(64), None),
    ]
    for call in calls:
        assert call() == cpdr.ERR_INVALID
        assert b"HOST_ONLY" in cpdr_lib.cpdr_last_error()
        assert call() == cpdr.ERR_INVALID
    for call in (lambda: L.cpdr_embed_fwd(None, P(16), 1, P(32), 4, 8, 1.0, P(48), None),
                 lambda: L.cpdr_embed_bwd_workspace_bytes(None, 1, 1, 8, ctypes.byref(ctypes.c_size_t()))):
        assert call() == cpdr.ERR_INVALID


@pytest.mark.parametrize("n,vocab,width,status", [
    (-1, 8, 8, cpdr.ERR_INVALID), ((1 << 30) + 1, 8, 8, cpdr.ERR_INVALID), (1, 0, 8, cpdr.ERR_INVALID),
    (1, (1 << 30) + 1, 8, cpdr.ERR_INVALID), (1, 8, 0, cpdr.ERR_INVALID), (1, 8, 12, cpdr.ERR_INVALID),
    (1, 8, (1 << 20) + 8, cpdr.ERR_UNSUPPORTED), (0, 1, 8, cpdr.OK), (1 << 30, 1 << 30, 8, cpdr.OK),
])
def test_embed_workspace_sizes(cpdr_lib, n, vocab, width, status):
    c, b = make(), ctypes.c_size_t()
    assert cpdr_lib.cpdr_embed_bwd_workspace_bytes(c._h, n, vocab, width, ctypes.byref(b)) == status
    if status == cpdr.OK:
        assert b.value >= 8 * n      # a list of positions and one of keys
        assert cpdr_lib.cpdr_embed_bwd_workspace_bytes(c._h, n, vocab, width, None) == cpdr.ERR_INVALID


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_tensors_that_are_not_on_the_gpu(cpdr_lib):
    c = make()
    calls = [
        lambda: c.layernorm_fwd(bf(3, 8), torch.ones(8), y=bf(3, 8)),
        lambda: c.layernorm_bwd(bf(3, 8), torch.ones(8), bf(3, 8)),
        lambda: c.embed_fwd(torch.zeros(3, dtype=torch.int32), bf(4, 8), bf(3, 8)),
        lambda: c.embed_bwd(torch.zeros(3, dtype=torch.int32), bf(3, 8), bf(4, 8)),
        lambda: c.delta_step(bf(3, 2, 64), bf(3, 2, 64), bf(3, 2, 64), bf(3, 2), torch.zeros(3, 2),
                             torch.zeros(5, 2, 64, 64), bf(3, 2, 64)),
        lambda: c.conv1d_step(bf(3, 8), torch.zeros(8, 4), None, bf(5, 3, 8), bf(3, 8)),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="must be on"):
            call()


def test_binding_refuses_wrong_shapes_and_dtypes(cpdr_lib):
    c = make()
    tok = torch.zeros(3, dtype=torch.int32)
    q, g, S = bf(3, 2, 64), torch.zeros(3, 2), torch.zeros(5, 2, 64, 64)
    bad = [
        (lambda: c.layernorm_fwd(bf(3, 8).float(), torch.ones(8), y=bf(3, 8)), "x must be"),
        (lambda: c.layernorm_bwd(bf(3, 8)[:, ::2], torch.ones(4), bf(3, 4)), "contiguous"),
        (lambda: c.embed_fwd(tok.long(), bf(4, 8), bf(3, 8)), "tokens must be"),
        (lambda: c.embed_fwd(tok, bf(8), bf(3, 8)), "table must be"),
        (lambda: c.embed_bwd(tok, bf(3, 8), bf(8)), "dtable must be"),
        (lambda: c.delta_step(q, q, q, bf(3, 2), g, S[..., :32], q.clone()), "state must be"),
        (lambda: c.delta_step(q, q, q, bf(3, 2), g, S.bfloat16(), q.clone()), "state must be"),
        (lambda: c.conv1d_step(bf(3, 8), torch.zeros(8, 4), None, bf(5, 8), bf(3, 8)), "state"),
        (lambda: c.conv1d_step(bf(3, 8), torch.zeros(8, 4), None, bf(5, 2, 8), bf(3, 8)), "state must be"),
    ]
    for call, what in bad:
        with pytest.raises(ValueError, match=what):
            call()
