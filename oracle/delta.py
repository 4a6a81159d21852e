"""The gated delta rule and layer norm in float64 NumPy, from their definitions: the rule token by token, and the
reverse of that recurrence for its gradients."""
from __future__ import annotations

import numpy as np


def _heads(x, Hv):
    """[Hk, n, d] as every value head reads it."""
    return np.repeat(x, Hv // x.shape[0], axis=0)


def delta_rule(q, k, v, g, beta, scale, W0=None):
    """One sequence: q, k [Hk, n, dk], v [Hv, n, dv], g, beta [Hv, n], W0 [Hv, dv, dk].  Returns (O, W_n)."""
    Hv, n, dv = v.shape
    q, k = _heads(q, Hv), _heads(k, Hv)
    W = np.zeros((Hv, dv, k.shape[2])) if W0 is None else W0.astype(np.float64).copy()
    O = np.zeros((Hv, n, dv))
    for t in range(n):
        W = np.exp(g[:, t])[:, None, None] * W
        e = v[:, t] - np.einsum("hvk,hk->hv", W, k[:, t])
        W = W + (beta[:, t, None] * e)[:, :, None] * k[:, t][:, None, :]
        O[:, t] = scale * np.einsum("hvk,hk->hv", W, q[:, t])
    return O, W


def delta_rule_backward(q, k, v, g, beta, scale, dO, W0=None, dWn=None):
    """Gradients of <O, dO> + <W_n, dWn>: (dq, dk [Hk, n, dk], dv, dg, dbeta, dW0)."""
    Hk, (Hv, n, dv) = q.shape[0], v.shape
    q, k = _heads(q, Hv), _heads(k, Hv)
    W = np.zeros((Hv, dv, k.shape[2])) if W0 is None else W0.astype(np.float64).copy()
    a = np.exp(g)
    before, errors, after = [], [], []
    for t in range(n):
        before.append(W)
        A = a[:, t, None, None] * W
        e = v[:, t] - np.einsum("hvk,hk->hv", A, k[:, t])
        W = A + (beta[:, t, None] * e)[:, :, None] * k[:, t][:, None, :]
        errors.append(e)
        after.append(W)
    dq, dk, dv_, dg, dbeta = (np.zeros_like(x, dtype=np.float64) for x in (q, k, v, g, beta))
    dW = np.zeros_like(W) if dWn is None else dWn.astype(np.float64).copy()
    for t in range(n - 1, -1, -1):
        dq[:, t] = scale * np.einsum("hvk,hv->hk", after[t], dO[:, t])
        dW = dW + scale * dO[:, t][:, :, None] * q[:, t][:, None, :]
        u = beta[:, t, None] * errors[t]
        du = np.einsum("hvk,hk->hv", dW, k[:, t])
        de = beta[:, t, None] * du
        dbeta[:, t] = (du * errors[t]).sum(-1)
        dv_[:, t] = de
        A = a[:, t, None, None] * before[t]
        dk[:, t] = np.einsum("hvk,hv->hk", dW, u) - np.einsum("hvk,hv->hk", A, de)
        dA = dW - de[:, :, None] * k[:, t][:, None, :]
        dg[:, t] = (A * dA).sum((-1, -2))
        dW = a[:, t, None, None] * dA
    fold = lambda x: x.reshape(Hk, Hv // Hk, n, x.shape[-1]).sum(1)
    return fold(dq), fold(dk), dv_, dg, dbeta, dW


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Rows x [rows, d]: (y, mean, rstd)."""
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(-1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    y = y if weight is None else y * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_backward(x, weight, dy, mean, rstd):
    """(dx, dweight, dbias)."""
    h = (x - mean[:, None]) * rstd[:, None]
    a = dy if weight is None else dy * weight
    dx = rstd[:, None] * (a - a.mean(-1, keepdims=True) - h * (a * h).mean(-1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)
