"""Pins of the oracle's selective scan, short convolution and root-mean-square norm: closed forms, torch's own layers,
central differences, and torch's rounding to e4m3."""
import numpy as np
import pytest
import torch

from oracle import inplace as orc
from oracle import scan as osc


def _inputs(H, G, n, P, N, seed=0):
    r = np.random.default_rng(seed)
    return [r.normal(size=(H, n, P)), r.normal(size=(H, n)), -r.uniform(0.2, 2.0, size=H), r.normal(size=(G, n, N)),
            r.normal(size=(G, n, N))]


def test_scalar_by_hand():
    """P = N = 1, decays 1 and 1/2: S1 = 0.5 * 2 * 3 = 3, o1 = 2 * 3; S2 = 1.5 + 1 * 1 * 4 = 5.5, o2 = 5.5 + D x."""
    x, B, C = np.array([[[2.0], [1.0]]]), np.array([[[3.0], [4.0]]]), np.array([[[2.0], [1.0]]])
    dt = np.array([[0.5, 1.0]])
    O, S = osc.selective_scan(x, dt, np.zeros(1), B, C)
    assert np.allclose(O[0, :, 0], [6.0, 7.0])
    O, S = osc.selective_scan(x, dt, np.array([-np.log(2.0)]), B, C, D=np.array([10.0]))
    assert np.allclose(O[0, :, 0], [26.0, 15.5]) and np.allclose(S, 5.5)


def test_scan_as_one_lower_triangular_product():
    """O = (C B^T exp(sums of A r)) r x: the whole sequence at once."""
    x, dt, A, B, C = _inputs(4, 2, 9, 3, 5)
    bias = np.array([0.1, -0.3, 0.0, 1.0])
    r = np.log1p(np.exp(dt + bias[:, None]))
    O, S = osc.selective_scan(x, dt, A, B, C, dt_bias=bias, softplus=True)
    for h in range(4):
        b = np.cumsum(A[h] * r[h])
        M = np.tril(C[h // 2] @ B[h // 2].T * np.exp(b[:, None] - b[None]))
        assert np.allclose(O[h], M @ (r[h][:, None] * x[h]))
        assert np.allclose(S[h], ((np.exp(b[-1] - b) * r[h])[:, None] * x[h]).T @ B[h // 2])


@pytest.mark.parametrize("softplus", [False, True])
def test_scan_backward_against_differences(softplus):
    H, G, n, P, N = 4, 2, 6, 3, 2
    x, dt, A, B, C = _inputs(H, G, n, P, N, 3)
    r = np.random.default_rng(4)
    D, bias, S0 = r.normal(size=H), r.normal(size=H), r.normal(size=(H, P, N))
    dO, dS = r.normal(size=x.shape), r.normal(size=S0.shape)
    args = {"x": x, "dt": dt, "A": A, "B": B, "C": C, "D": D, "dt_bias": bias, "S0": S0}
    d = osc.selective_scan_backward(x, dt, A, B, C, dO, D, bias, softplus, S0, dS)

    def loss(**kw):
        O, S = osc.selective_scan(softplus=softplus, **{**args, **kw})
        return (O * dO).sum() + (S * dS).sum()

    for name, v in args.items():
        step = r.normal(size=v.shape)
        e = 1e-5
        diff = (loss(**{name: v + e * step}) - loss(**{name: v - e * step})) / (2 * e)
        assert np.isclose(diff, (d["d" + name] * step).sum(), rtol=1e-6, atol=1e-8), name


def test_scan_resumes():
    x, dt, A, B, C = _inputs(2, 1, 9, 4, 3)
    cut = lambda a, b: (x[:, a:b], dt[:, a:b], A, B[:, a:b], C[:, a:b])
    O, S = osc.selective_scan(*cut(0, 9))
    Oa, Sa = osc.selective_scan(*cut(0, 4))
    Ob, Sb = osc.selective_scan(*cut(4, 9), S0=Sa)
    assert np.allclose(np.concatenate([Oa, Ob], 1), O) and np.allclose(Sb, S)


@pytest.mark.parametrize("K", [1, 2, 4, 8])
def test_convolution(K):
    r = np.random.default_rng(K)
    x, w, b, x0 = r.normal(size=(11, 5)), r.normal(size=(5, K)), r.normal(size=5), r.normal(size=(K - 1, 5))
    y, last = osc.short_conv(x, w, b, False)
    assert np.allclose(y, orc.causal_depthwise_conv1d(x, w) + b)
    t = torch.nn.functional.conv1d(torch.tensor(np.concatenate([x0, x]).T)[None], torch.tensor(w)[:, None], torch.tensor(b),
                                   groups=5)
    y, last = osc.short_conv(x, w, b, True, x0)
    assert np.allclose(y, torch.nn.functional.silu(t)[0].T.numpy())
    assert np.allclose(last, np.concatenate([x0, x])[11:])
    # shorter than the taps: earlier rows stay among the last ones
    assert np.allclose(osc.short_conv(x[:1], w, b, True, x0)[1], np.concatenate([x0, x[:1]])[1:])


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("n", [1, 2, 7])
def test_convolution_backward_against_differences(n, silu):
    r = np.random.default_rng(n)
    d, K = 3, 4
    args = {"x": r.normal(size=(n, d)), "w": r.normal(size=(d, K)), "bias": r.normal(size=d), "x0": r.normal(size=(K - 1, d))}
    dy, dl = r.normal(size=(n, d)), r.normal(size=(K - 1, d))
    grads = dict(zip(("x", "w", "bias", "x0"), osc.short_conv_backward(args["x"], args["w"], dy, args["bias"], silu,
                                                                      args["x0"], dl)))

    def loss(**kw):
        y, last = osc.short_conv(silu=silu, **{**args, **kw})
        return (y * dy).sum() + (last * dl).sum()

    for name, v in args.items():
        step = r.normal(size=v.shape)
        diff = (loss(**{name: v + 1e-5 * step}) - loss(**{name: v - 1e-5 * step})) / 2e-5
        assert np.isclose(diff, (grads[name] * step).sum(), rtol=1e-6, atol=1e-8), name


def test_rms_norm():
    r = np.random.default_rng(0)
    h, w, dy, dh = r.normal(size=(4, 9)), r.normal(size=9), r.normal(size=(4, 9)), r.normal(size=(4, 9))
    t = [torch.tensor(v, requires_grad=True) for v in (h, w)]
    y = torch.nn.functional.rms_norm(t[0], (9,), t[1], 1e-3)
    out, rstd = osc.rms_norm(h, w, 1e-3)
    assert np.allclose(out, y.detach().numpy())
    ((y * torch.tensor(dy)).sum() + (t[0] * torch.tensor(dh)).sum()).backward()
    dx, dw = osc.rms_norm_backward(h, w, dy, rstd, dh)
    assert np.allclose(dx, t[0].grad.numpy()) and np.allclose(dw, t[1].grad.numpy())


def test_e4m3_and_scales():
    v = np.concatenate([np.linspace(-448, 448, 4001), 2.0 ** np.linspace(-14, 8, 999), [0.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    assert np.array_equal(osc.e4m3(v), torch.tensor(v).to(torch.float8_e4m3fn).double().numpy())
    y = np.array([[1.0, -896.0, 0.0, 0.0, 4.48]])
    assert np.allclose(osc.scales(y, 2), [[2.0, 2.0 ** -126, 0.01]]) and np.allclose(osc.scales(y), [[2.0]])
