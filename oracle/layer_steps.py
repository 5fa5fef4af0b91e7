"""fp64 oracle of the layer steps around the token mixers: the gated linear
recurrence, the RMS norm and the matrix product with its epilogue, with their
gradients.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle``: the CUDA library
shares nothing with it.  Everything is written token by token or row by row
from the definitions, in sequence order (the zigzag memory order is undone by
the caller with ``oracle.layout``).  Each function also returns how far a
computation in fp32 may be off: the roundings along its path, added up in
absolute values (derived at each place).
"""
from __future__ import annotations

import math

import numpy as np

U32 = 2.0 ** -24                      # half a step of fp32, relative
HALF_STEP = {"fp32": U32, "bf16": 2.0 ** -8}


def as64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def bounds_of(B, T, cu_seqlens=None):
    """(row, first, end) of every sequence."""
    if cu_seqlens is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(v) for v in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    return [(0, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]


# Relative rounding of one token's step: exp in fp32 (one unit in the last
# place, 2 U32, and the same again for its argument's own reduction), the
# product and sum (one rounding each), and as many again for the products of
# maps (A2 A1, A2 B1 + B2) that carry a state across groups: 8 U32.
STEP = 8 * U32


def glr_forward(x, g, h0=None, cu_seqlens=None):
    """h_t = exp(g_t) h_{t-1} + x_t.  x, g [B, T, C]; h0 [N, C].

    Returns y [B, T, C], hT [N, C], the states before each token, and the
    error bounds of y and hT: with H the same recurrence on absolute values,
    E_t = a_t (E_{t-1} + STEP H_{t-1}) + STEP |x_t|."""
    x, g, h0 = as64(x), as64(g), as64(h0)
    B, T, C = x.shape
    seqs = bounds_of(B, T, cu_seqlens)
    y, prev, err, mag = (np.zeros_like(x) for _ in range(4))
    hT, eT = np.zeros((len(seqs), C)), np.zeros((len(seqs), C))
    with np.errstate(under="ignore"):
        for n, (b, s, e) in enumerate(seqs):
            h = np.zeros(C) if h0 is None else h0[n].copy()
            H, E = np.abs(h), np.zeros(C)
            for t in range(s, e):
                a = np.exp(g[b, t])
                prev[b, t], mag[b, t], err[b, t] = h, H, E
                h = a * h + x[b, t]
                E = a * (E + STEP * H) + STEP * np.abs(x[b, t])
                H = a * H + np.abs(x[b, t])
                y[b, t] = h
            hT[n], eT[n] = h, E
    # y's own error is that of the state behind the token
    ey = np.zeros_like(x)
    for n, (b, s, e) in enumerate(seqs):
        if e > s:
            ey[b, s:e - 1], ey[b, e - 1] = err[b, s + 1:e], eT[n]
    return dict(y=y, hT=hT, prev=prev, mag=mag, e_prev=err, e_y=ey, e_hT=eT)


def glr_backward(x, g, dy, h0=None, dhT=None, cu_seqlens=None):
    """Gradients of sum <dy, y> + sum <dhT, hT>: dx, dg [B, T, C], dh0 [N, C],
    with their error bounds (e_dx, e_dg, e_dh0)."""
    f = glr_forward(x, g, h0, cu_seqlens)
    x, g, dy, dhT = as64(x), as64(g), as64(dy), as64(dhT)
    B, T, C = x.shape
    seqs = bounds_of(B, T, cu_seqlens)
    dx, dg, e_dx, e_dg = (np.zeros_like(x) for _ in range(4))
    dh0, e_dh0 = np.zeros((len(seqs), C)), np.zeros((len(seqs), C))
    with np.errstate(under="ignore"):
        for n, (b, s, e) in enumerate(seqs):
            q = np.zeros(C) if dhT is None else dhT[n].copy()    # a_{t+1} dh_{t+1}
            Q, E = np.abs(q), np.zeros(C)
            for t in range(e - 1, s - 1, -1):
                a = np.exp(g[b, t])
                dh, D = dy[b, t] + q, np.abs(dy[b, t]) + Q
                Ed = E + STEP * D
                q, Q, E = a * dh, a * D, a * (Ed + STEP * D)
                dx[b, t], e_dx[b, t] = dh, Ed
                dg[b, t] = q * f["prev"][b, t]
                e_dg[b, t] = E * f["mag"][b, t] + Q * f["e_prev"][b, t] + STEP * Q * f["mag"][b, t]
            dh0[n], e_dh0[n] = q, E
    return dict(dx=dx, dg=dg, dh0=dh0, e_dx=e_dx, e_dg=e_dg, e_dh0=e_dh0)


def glr_steps(x, g, state, slots):
    """Rows one after the other over a pool of states; y is nan where a row does nothing."""
    x, g, state = as64(x), as64(g), as64(state).copy()
    y = np.full_like(x, np.nan)
    for i, s in enumerate(slots):
        if 0 <= s < state.shape[0]:
            state[s] = np.exp(g[i]) * state[s] + x[i]
            y[i] = state[s]
    return y, state


# Rows of up to 16384 elements are summed by threads of at most 32 elements,
# then over at most 37 partial sums: under 80 roundings, half of that after
# the square root, and a few for rsqrt and the products around it.
ROW = 64 * U32


def rmsnorm_forward(x, weight, eps, residual=None):
    """x [rows, width] -> s, y (with the relative error bound ROW of y)."""
    x, w = as64(x), as64(weight)
    s = x if residual is None else x + as64(residual)
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return dict(s=s, y=s * rstd * w)


def e4m3_scale(y):
    return np.maximum(np.abs(y).max(axis=1) / 448.0, 2.0 ** -126)


def rmsnorm_backward(s, weight, eps, dy, dsum=None):
    """ds [rows, width], dweight [width] and their absolute error bounds: each
    term's magnitude times the roundings that it passes (a row's sums, ROW;
    the sum over rows, one rounding per row)."""
    s, w, dy = as64(s), as64(weight), as64(dy)
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    wdy = w * dy
    ds = rstd * (wdy - s * rstd ** 2 * (s * wdy).mean(axis=1, keepdims=True))
    mag = rstd * (np.abs(wdy) + np.abs(s) * rstd ** 2 * np.abs(s * wdy).mean(axis=1, keepdims=True))
    if dsum is not None:
        ds, mag = ds + as64(dsum), mag + np.abs(as64(dsum))
    t = dy * s * rstd
    return dict(ds=ds, dweight=t.sum(axis=0), e_ds=2 * ROW * mag,
                e_dweight=(ROW + (s.shape[0] + 32) * U32) * np.abs(t).sum(axis=0))


def _erf(x):
    return np.vectorize(math.erf, otypes=[np.float64])(x)


def activation(z, act):
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    return z


def activation_grad(z, act):
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


# A sum of n products in fp32: the tensor cores add 16 (bf16) or 32 (e4m3)
# exact products at once to the running sum, each time with an error of at most
# one unit in the last place (2 U32; they may cut instead of rounding) of what
# the absolute values add up to; 16 more for the roundings inside an addition
# and for the sums of a split.
def _sum_error(n):
    return (n / 16 + 16) * 2 * U32


# exp, the quotient or erf, and the products around them, in fp32: 16 U32 of
# what the value is made of (z act terms of size |z|, gradients of size 1 + |z|).
ACT = 16 * U32


def linear_forward(x, w, bias=None, act=None, residual=None, x_scale=None, w_scale=None):
    """z = (x w^T) x_scale w_scale + bias, y = act(z) + residual, and the
    error bounds of both (|act'| is at most 1.13)."""
    x, w = as64(x), as64(w)
    z, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if x_scale is not None:
        s = as64(x_scale)[:, None] * as64(w_scale)[None, :]
        z, mag = z * s, mag * s
    e_z = mag * (_sum_error(x.shape[1]) + 4 * U32)
    if bias is not None:
        z = z + as64(bias)
        e_z = e_z + 2 * U32 * np.abs(z)
    y, e_y = activation(z, act), 1.13 * e_z + ACT * np.abs(z)
    if residual is not None:
        y = y + as64(residual)
        e_y = e_y + 2 * U32 * np.abs(y)
    return dict(z=z, y=y, e_z=e_z, e_y=e_y)


def linear_backward(x, w, dy, z=None, act=None):
    """dx, dw, dbias and their error bounds: dz is an operand rounded to bf16
    (half a step of each value), dbias a sum of unrounded values."""
    x, w, dy = as64(x), as64(w), as64(dy)
    if act in ("silu", "gelu"):
        z = as64(z)
        dz, e = dy * activation_grad(z, act), ACT * np.abs(dy) * (1 + np.abs(z))
    else:
        dz, e = dy, np.zeros_like(dy)
    step = HALF_STEP["bf16"] * np.abs(dz) + e if act in ("silu", "gelu") else e
    rows, N = dz.shape
    A = np.abs(dz) + step
    return dict(dx=dz @ w, dw=dz.T @ x, dbias=dz.sum(0),
                e_dx=step @ np.abs(w) + _sum_error(N) * (A @ np.abs(w)),
                e_dw=step.T @ np.abs(x) + _sum_error(rows) * (A.T @ np.abs(x)),
                e_dbias=e.sum(0) + (rows + 32) * U32 * np.abs(dz).sum(0))
