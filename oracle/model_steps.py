"""fp64 oracle of the steps of a delta-rule model beside its mixers and in
decoding: the delta rule and the causal conv token by token over pools of
slots, the layer norm and the embedding, with their gradients.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle``: written row by row from
the definitions.  Each function also returns how far a computation in fp32 may
be off: the roundings along its path, derived at each place.
"""
from __future__ import annotations

import numpy as np

from .layer_steps import ROW, U32, as64


def delta_steps(q, k, v, beta, g, state, slots, scale=1.0):
    """Rows one after the other over a pool of states [S, H, dk, dv]:
        S <- (I - beta k k^T) Diag(exp g) S + beta k v^T,   o = scale S^T q.

    Returns o (nan where a row does nothing), the states and error bounds:
    e_o for each output, e_state [S, H, dv] for the 2-norm of each value dim's
    column.  A column's error passes (I - beta k k^T) Diag(a), whose norm is at
    most max(1, |1 - beta |k|^2|) max a; a token adds, in norms of the column P
    behind the gate: 5 U32 |P| (exp, 4 U32, and its product), a dot product of
    up to 19 roundings along a path (of 128 key dims 16 multiply-adds in a lane
    and three sums over lanes; where a lane has four of them, 3 and five), 19 U32
    |k| |P| (Cauchy), times beta |k|, three roundings of beta (v - .) k and one of
    the new column.  An output: 19 of P^T q and one of adding (q . k) D, whose own
    are fewer (3 and five, one of D); the scale's is half a step of fp32 at most,
    which the output's type adds."""
    q, k, v, beta, g, state = (as64(t) for t in (q, k, v, beta, g, state))
    state = state.copy()
    n, H, d = k.shape
    G = q.shape[1] // H
    o, e_o = np.full(q.shape[:2] + v.shape[2:], np.nan), np.zeros(q.shape[:2] + v.shape[2:])
    E = np.zeros((state.shape[0], H, v.shape[2]))
    for i, s in enumerate(slots):
        if not 0 <= s < state.shape[0]:
            continue
        for h in range(H):
            a = np.exp(g[i, h]) * np.ones(d)
            P = a[:, None] * state[s, h]
            kk, b = np.linalg.norm(k[i, h]), abs(beta[i, h])
            c = np.linalg.norm(P, axis=0)
            x = v[i, h] - P.T @ k[i, h]
            state[s, h] = P + beta[i, h] * np.outer(k[i, h], x)
            new = np.linalg.norm(state[s, h], axis=0)
            E[s, h] = (max(1.0, abs(1 - beta[i, h] * kk * kk)) * a.max() * E[s, h]
                       + U32 * (5 * c + 19 * b * kk * kk * c + 3 * b * kk * np.abs(x) + new))
            for j in range(h * G, (h + 1) * G):
                qq = np.linalg.norm(q[i, j])
                o[i, j] = scale * (state[s, h].T @ q[i, j])
                # the sum may be taken over P, the new term added: P^T q + (q . k) D
                e_o[i, j] = abs(scale) * qq * (E[s, h] + U32 * 20 * (c + new + b * kk * np.abs(x)))
    return dict(o=o, state=state, e_o=e_o, e_state=E)


def conv_steps(x, weight, bias, state, slots, activation="silu"):
    """Rows one after the other over a pool of windows [S, W - 1, C].

    e_y: W + 2 roundings of the sum's absolute value; SiLU's fast exponential is
    off by 4 U32 and by its argument's rounding, 4 U32 |z|, and its quotient by
    4 U32 (all times |z|; |silu'| is at most 1.1)."""
    x, w, state = as64(x), as64(weight), as64(state).copy()
    b = np.zeros(x.shape[1]) if bias is None else as64(bias)
    W = w.shape[1]
    y, e_y = np.full_like(x, np.nan), np.zeros_like(x)
    for i, s in enumerate(slots):
        if not 0 <= s < state.shape[0]:
            continue
        win = np.concatenate([state[s], x[i:i + 1]])
        z = b + (win * w.T).sum(0)
        e = (W + 2) * U32 * (np.abs(b) + np.abs(win * w.T).sum(0))
        if activation == "silu":
            e = 1.1 * e + (8 + 4 * np.abs(z)) * U32 * np.abs(z)
            z = z / (1.0 + np.exp(-z))
        y[i], e_y[i] = z, e
        state[s] = win[1:]
    return dict(y=y, state=state, e_y=e_y)


def _centred(s, eps):
    c = s - s.mean(axis=1, keepdims=True)
    return c, 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)


def _centre_error(s, c, summed):
    """How far a difference to the mean may be off: the first mean is off by a
    row's sum, ROW mean|s|; the differences to it, each rounded twice, are
    corrected by their own mean, another row's sum (ROW) of them; and, where s is
    a sum itself, that one's rounding."""
    first = ROW * np.abs(s).mean(axis=1, keepdims=True)
    return (3 * U32 * (np.abs(c) + first) + ROW * (np.abs(c).mean(axis=1, keepdims=True) + first)
            + (2 * U32 * np.abs(s) if summed else 0.0))


def layernorm_forward(x, weight, bias, eps, residual=None):
    """x [rows, width] -> s, y and y's error bound."""
    x, w = as64(x), as64(weight)
    b = np.zeros_like(w) if bias is None else as64(bias)
    s = x if residual is None else x + as64(residual)
    c, rstd = _centred(s, eps)
    y = c * rstd * w + b
    e = np.abs(w) * rstd * (_centre_error(s, c, residual is not None) + ROW * np.abs(c))
    return dict(s=s, y=y, e_y=e + 2 * U32 * (np.abs(b) + np.abs(y)))


def layernorm_backward(s, weight, eps, dy, dsum=None):
    """ds [rows, width], dweight and dbias [width] and their error bounds."""
    s, w, dy = as64(s), as64(weight), as64(dy)
    c, rstd = _centred(s, eps)
    xh, u = c * rstd, w * dy
    e_xh = rstd * _centre_error(s, c, False) + ROW * np.abs(xh)
    mu, dot = u.mean(axis=1, keepdims=True), (u * xh).mean(axis=1, keepdims=True)
    ds = rstd * (u - mu - xh * dot)
    a = np.abs(u)
    mag = a + a.mean(axis=1, keepdims=True)
    e_dot = ROW * (np.abs(u * xh).mean(axis=1, keepdims=True)) + (a * e_xh).mean(axis=1, keepdims=True)
    e = rstd * (2 * ROW * mag + 2 * e_xh * np.abs(dot) + 2 * np.abs(xh) * e_dot) + ROW * np.abs(ds)
    if dsum is not None:
        ds = ds + as64(dsum)
    e = e + 2 * U32 * np.abs(ds)
    sums = (s.shape[0] + 32) * U32
    return dict(ds=ds, dweight=(dy * xh).sum(0), dbias=dy.sum(0), e_ds=e,
                e_dweight=(np.abs(dy) * e_xh).sum(0) + sums * np.abs(dy * xh).sum(0), e_dbias=sums * np.abs(dy).sum(0))


def embed_backward(tokens, dy, vocab, scale=1.0):
    """dtable [vocab, D]; a token's sum has one rounding per row, and one of the scale."""
    dy = as64(dy)
    out, mag, count = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1])), np.zeros((vocab, 1))
    for i, t in enumerate(np.asarray(tokens).tolist()):
        if 0 <= t < vocab:
            out[t] += dy[i]
            mag[t] += np.abs(dy[i])
            count[t] += 1
    return dict(dtable=scale * out, e_dtable=(count + 2) * U32 * abs(scale) * mag)
