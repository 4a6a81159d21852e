"""The selective scan, its short convolution and the root-mean-square norm in float64 NumPy, from their definitions: the
scan token by token, and the reverse of that recurrence for its gradients."""
from __future__ import annotations

import numpy as np


def rates(dt, dt_bias=None, softplus=False):
    """The rates of tokens [H, n] (or [..., H] turned by the caller) and their derivative by dt."""
    x = dt if dt_bias is None else dt + np.reshape(dt_bias, (-1, 1))
    return (np.logaddexp(x, 0.0), 1 / (1 + np.exp(-x))) if softplus else (x, np.ones_like(x))


def _heads(t, H):
    """[G, n, N] as every head reads it."""
    return np.repeat(t, H // t.shape[0], axis=0)


def selective_scan(x, dt, A, B, C, D=None, dt_bias=None, softplus=False, S0=None):
    """One sequence: x [H, n, P], dt [H, n], A, D, dt_bias [H], B, C [G, n, N], S0 [H, P, N].  Returns (O, S_n)."""
    H, n, P = x.shape
    B, C = _heads(B, H), _heads(C, H)
    r = rates(dt, dt_bias, softplus)[0]
    S = np.zeros((H, P, B.shape[2])) if S0 is None else S0.astype(np.float64).copy()
    O = np.zeros((H, n, P))
    for t in range(n):
        S = np.exp(A * r[:, t])[:, None, None] * S + (r[:, t, None] * x[:, t])[:, :, None] * B[:, t][:, None, :]
        O[:, t] = np.einsum("hpn,hn->hp", S, C[:, t])
    return O if D is None else O + D[:, None, None] * x, S


def selective_scan_backward(x, dt, A, B, C, dO, D=None, dt_bias=None, softplus=False, S0=None, dSn=None):
    """Gradients of <O, dO> + <S_n, dSn>: a dict of dx, ddt, dA, dB, dC, dD, ddt_bias, dS0."""
    G, (H, n, P) = B.shape[0], x.shape
    B, C = _heads(B, H), _heads(C, H)
    r, slope = rates(dt, dt_bias, softplus)
    a = np.exp(A[:, None] * r)
    S = np.zeros((H, P, B.shape[2])) if S0 is None else S0.astype(np.float64).copy()
    states = [S]
    for t in range(n):
        S = a[:, t, None, None] * S + (r[:, t, None] * x[:, t])[:, :, None] * B[:, t][:, None, :]
        states.append(S)
    dx, dB, dC, dr, dlog = np.zeros_like(x), np.zeros_like(B), np.zeros_like(C), np.zeros_like(r), np.zeros_like(r)
    dS = np.zeros_like(S) if dSn is None else dSn.astype(np.float64).copy()
    for t in range(n - 1, -1, -1):
        dC[:, t] = np.einsum("hpn,hp->hn", states[t + 1], dO[:, t])
        dS = dS + dO[:, t][:, :, None] * C[:, t][:, None, :]
        du = np.einsum("hpn,hn->hp", dS, B[:, t])
        dB[:, t] = np.einsum("hpn,hp->hn", dS, r[:, t, None] * x[:, t])
        dx[:, t] = r[:, t, None] * du
        dr[:, t] = (du * x[:, t]).sum(-1)
        dlog[:, t] = a[:, t] * (dS * states[t]).sum((1, 2))
        dS = a[:, t, None, None] * dS
    ddt = (dr + A[:, None] * dlog) * slope
    fold = lambda t: t.reshape(G, H // G, n, t.shape[-1]).sum(1)
    return {"dx": dx if D is None else dx + D[:, None, None] * dO, "ddt": ddt, "dA": (dlog * r).sum(1), "dB": fold(dB),
            "dC": fold(dC), "dD": (dO * x).sum((1, 2)), "ddt_bias": ddt.sum(1), "dS0": dS}


def _silu(z):
    return z / (1 + np.exp(-z))


def short_conv(x, w, bias=None, silu=True, x0=None):
    """One sequence: x [n, d], w [d, K], x0 [K - 1, d].  Returns (y [n, d], the last K - 1 rows of x0 and x)."""
    (n, d), K = x.shape, w.shape[1]
    line = np.concatenate([np.zeros((K - 1, d)) if x0 is None else x0, x])
    z = np.zeros((n, d)) if bias is None else np.tile(np.asarray(bias, dtype=np.float64), (n, 1))
    for t in range(n):
        z[t] += (line[t:t + K] * w.T).sum(0)
    return _silu(z) if silu else z, line[n:]


def short_conv_backward(x, w, dy, bias=None, silu=True, x0=None, dx_final=None):
    """Gradients of <y, dy> + <last rows, dx_final>: (dx, dw, dbias, dx0)."""
    (n, d), K = x.shape, w.shape[1]
    line = np.concatenate([np.zeros((K - 1, d)) if x0 is None else x0, x])
    dline, dw, db = np.zeros((n + K - 1, d)), np.zeros((d, K)), np.zeros(d)
    if dx_final is not None:
        dline[n:] += dx_final
    z = short_conv(x, w, bias, False, x0)[0]
    for t in range(n):
        s = 1 / (1 + np.exp(-z[t]))
        dz = dy[t] * (s * (1 + z[t] * (1 - s)) if silu else 1.0)
        dline[t:t + K] += dz * w.T
        dw += (dz * line[t:t + K]).T
        db += dz
    return dline[K - 1:], dw, db, dline[:K - 1]


def rms_norm(h, weight=None, eps=1e-5):
    """Rows h [rows, d]: (y, 1 / sqrt(mean(h^2) + eps))."""
    rstd = 1.0 / np.sqrt((h ** 2).mean(-1) + eps)
    y = h * rstd[:, None]
    return (y if weight is None else y * weight), rstd


def rms_norm_backward(h, weight, dy, rstd, dh=None):
    """(dx, dweight)."""
    n = h * rstd[:, None]
    a = dy if weight is None else dy * weight
    dx = rstd[:, None] * (a - n * (a * n).mean(-1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * n).sum(0)


def e4m3(v):
    """The e4m3 value nearest to each of v, |v| <= 448: 3 bits behind the point, exponents from -6, ties to even."""
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -20))), -6) - 3)
    return np.round(v / step) * step


def scales(y, group=None):
    """y [rows, d] in groups of columns: max |y| / 448, at least 2^-126, [rows, groups]."""
    group = group or y.shape[1]
    parts = [np.abs(y[:, i:i + group]).max(-1) for i in range(0, y.shape[1], group)]
    return np.maximum(np.stack(parts, -1) / 448.0, 2.0 ** -126)
