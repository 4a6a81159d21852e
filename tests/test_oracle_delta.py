"""Pins of the oracle's gated delta rule and layer norm: closed forms, torch's autograd of torch-built layers in
fp64, and central differences."""
import numpy as np
import pytest
import torch

from oracle import delta as od


def _inputs(Hk, Hv, n, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    k = r.normal(size=(Hk, n, dk))
    return (r.normal(size=(Hk, n, dk)), k / np.linalg.norm(k, axis=-1, keepdims=True), r.normal(size=(Hv, n, dv)),
            -r.exponential(0.3, size=(Hv, n)), r.uniform(0.1, 1.0, size=(Hv, n)))


def test_orthonormal_keys_without_decay_store_and_return_the_values():
    """With beta = 1, no decay and orthonormal keys each token's value is stored exactly, and the query of a past key
    returns it."""
    r = np.random.default_rng(1)
    n = 6
    k = np.eye(n)[None]
    v = r.normal(size=(1, n, 5))
    O, W = od.delta_rule(k, k, v, np.zeros((1, n)), np.ones((1, n)), 1.0)
    assert np.allclose(O, v)
    assert np.allclose(W[0], v[0].T)
    # writing a key again replaces its value
    O, W = od.delta_rule(np.tile(k[:, :1], (1, 2, 1)), np.tile(k[:, :1], (1, 2, 1)), v[:, :2], np.zeros((1, 2)),
                         np.ones((1, 2)), 1.0)
    assert np.allclose(W[0][:, 0], v[0, 1]) and np.allclose(W[0][:, 1:], 0)


def test_scalar_by_hand():
    """dk = dv = 1: W1 = 1 * 0.5 * 2 = 1; then decay 0.5: 0.5, error 3 - 0.5 * 2 = 2, W2 = 0.5 + 0.25 * 2 * 2 = 1.5."""
    q = np.array([[[1.0], [2.0]]])
    k = np.array([[[1.0], [2.0]]])
    v = np.array([[[2.0], [3.0]]])
    O, W = od.delta_rule(q, k, v, np.log([[1.0, 0.5]]), np.array([[0.5, 0.25]]), 2.0)
    assert np.allclose(O[0, :, 0], [2.0, 6.0]) and np.allclose(W, 1.5)


def test_reset_and_resume():
    q, k, v, g, beta = _inputs(1, 2, 9, 4, 3)
    O, W = od.delta_rule(q, k, v, g, beta, 0.7)
    Oa, Wa = od.delta_rule(q[:, :4], k[:, :4], v[:, :4], g[:, :4], beta[:, :4], 0.7)
    Ob, Wb = od.delta_rule(q[:, 4:], k[:, 4:], v[:, 4:], g[:, 4:], beta[:, 4:], 0.7, Wa)
    assert np.allclose(np.concatenate([Oa, Ob], 1), O) and np.allclose(Wb, W)
    g[:, 4] = -np.inf
    O, W = od.delta_rule(q, k, v, g, beta, 0.7)
    Ob, Wb = od.delta_rule(q[:, 4:], k[:, 4:], v[:, 4:], g[:, 4:], beta[:, 4:], 0.7)
    assert np.allclose(O[:, 4:], Ob) and np.allclose(W, Wb)


@pytest.mark.parametrize("start", [False, True])
def test_backward_against_autograd_and_differences(start):
    Hk, Hv, n, dk, dv = 2, 4, 7, 3, 5
    q, k, v, g, beta = _inputs(Hk, Hv, n, dk, dv, 3)
    r = np.random.default_rng(4)
    dO, W0, dWn = r.normal(size=(Hv, n, dv)), r.normal(size=(Hv, dv, dk)), r.normal(size=(Hv, dv, dk))
    grads = od.delta_rule_backward(q, k, v, g, beta, 0.6, dO, W0 if start else None, dWn if start else None)
    x = [torch.tensor(t, requires_grad=True) for t in (q, k, v, g, beta, W0 if start else np.zeros_like(W0))]
    tq, tk, tv, tg, tb, W = x
    tq, tk = (t.repeat_interleave(Hv // Hk, 0) for t in (tq, tk))
    O = []
    for t in range(n):
        W = W * tg[:, t].exp()[:, None, None]
        e = tv[:, t] - (W * tk[:, t, None]).sum(-1)
        W = W + (tb[:, t, None] * e)[..., None] * tk[:, t, None]
        O.append(0.6 * (W * tq[:, t, None]).sum(-1))
    loss = (torch.stack(O, 1) * torch.tensor(dO)).sum() + ((W * torch.tensor(dWn)).sum() if start else 0)
    for a, b in zip(grads, torch.autograd.grad(loss, x)):
        assert np.allclose(a, b.numpy(), atol=1e-12)

    def value(args):
        O, W = od.delta_rule(*args[:5], 0.6, args[5])
        return (O * dO).sum() + ((W * dWn).sum() if start else 0.0)
    args = [q, k, v, g, beta, W0 if start else np.zeros_like(W0)]
    for i, a in enumerate(args):
        at = tuple(s // 2 for s in a.shape)
        d = []
        for e in (1e-6, -1e-6):
            b = [t.copy() for t in args]
            b[i][at] += e
            d.append(value(b))
        assert abs((d[0] - d[1]) / 2e-6 - grads[i][at]) < 1e-7


def test_layer_norm_against_torch():
    r = np.random.default_rng(5)
    x, w, b, dy = r.normal(3, 2, size=(5, 7)), r.normal(size=7), r.normal(size=7), r.normal(size=(5, 7))
    y, mean, rstd = od.layer_norm(x, w, b, 1e-3)
    t = [torch.tensor(a, requires_grad=True) for a in (x, w, b)]
    ref = torch.nn.functional.layer_norm(t[0], (7,), t[1], t[2], 1e-3)
    assert np.allclose(y, ref.detach().numpy())
    grads = od.layer_norm_backward(x, w, dy, mean, rstd)
    for a, e in zip(grads, torch.autograd.grad((ref * torch.tensor(dy)).sum(), t)):
        assert np.allclose(a, e.numpy())
