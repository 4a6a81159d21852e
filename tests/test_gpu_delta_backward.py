"""The gated delta rule's backward on the GPU against the oracle's reverse recurrence in fp64.

Tolerances (relative Frobenius norm; a rounding to bf16 is off by at most 2^-8 of the value, fp32 2^-24).
  bf16 dv          X is made from pairs of bf16 values (2^-16) and rounded once: 2^-8, and 2 sqrt(5) 2^-16.
  bf16 dq, dk      between the inputs and them lie, in a chain, the roundings of the state or its gradient, of E or X, of
                   Mq or Mk, of dO S^T's operands and of the result: at most 5 independent ones, sqrt(5) 2^-8; dk sums
                   four such products of like size, some of which cancel: taken twice.
  bf16 dg, dbeta   dots of the same quantities, sums of terms that cancel in part: as dk.
  bf16 dW_init     pairs of bf16 values as the forward's final state: 2 sqrt(5) 2^-16.
  fp32             sums of at most dk + dv + 128 <= 512 terms, twice in a chain: 1024 * 2^-24.
A sequence of one or two tokens has dg (and a part of dk) that is exactly zero in the reference; what is left is held to
the same tolerance of the largest gradient there is.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import delta as od
from test_gpu_delta import f64, make

pytestmark = pytest.mark.gpu

B16, F32 = torch.bfloat16, torch.float32
CHAIN = 2 * 5 ** 0.5 * 2.0 ** -16
TOL = {B16: dict(dq=5 ** 0.5 * 2.0 ** -8, dk=2 * 5 ** 0.5 * 2.0 ** -8, dv=2.0 ** -8 + CHAIN, dg=2 * 5 ** 0.5 * 2.0 ** -8,
                 dbeta=2 * 5 ** 0.5 * 2.0 ** -8, dW_init=CHAIN),
       F32: dict.fromkeys(("dq", "dk", "dv", "dg", "dbeta", "dW_init"), 1024 * 2.0 ** -24)}
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dW_init")


def check(got, ref, dtype, what=""):
    for name, a, b in zip(NAMES, got, ref):
        if a is None:
            continue
        a = a.double().cpu().numpy()
        n = np.linalg.norm(b)
        err = np.linalg.norm(a - b) / n if n > 1e-12 else np.abs(a).max(initial=0.0)
        print("  ", what, name, err, flush=True)
        assert err <= TOL[dtype][name], (what, name)


def extras(rows, Hv, n, dk, dv, dtype, layout, seed=3):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    dO = r(rows, n, Hv, dv).to(dtype).cuda().transpose(1, 2)
    return (dO if layout == "token" else dO.contiguous(), r(rows, Hv, dv, dk).mul(0.3).cuda(),
            r(rows, Hv, dv, dk).mul(0.3).cuda())


CASES = [  # B, Hk, Hv, n, dk, dv, layout
    (1, 1, 1, 3, 64, 16, "head"),
    (2, 2, 4, 63, 64, 72, "token"),
    (1, 2, 2, 64, 128, 128, "head"),
    (1, 1, 3, 200, 16, 8, "token"),
    (1, 2, 4, 130, 96, 80, "head"),
    (1, 1, 2, 257, 256, 40, "token"),
    (3, 1, 1, 65, 8, 24, "token"),
    (1, 1, 2, 330, 128, 136, "token"),
    (1, 3, 3, 150, 200, 200, "head"),
]


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("start", [False, True])
def test_gradients(case, dtype, start):
    B, Hk, Hv, n, dk, dv, layout = case
    print("delta backward", case, dtype, start, flush=True)
    args = make(B, Hk, Hv, n, dk, dv, dtype, layout)
    dO, W0, dWn = extras(B, Hv, n, dk, dv, dtype, layout)
    if not start:
        W0 = dWn = None
    got = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, scale=0.4, W_init=W0)
    assert all(a.stride() == b.stride() and a.dtype == dtype for a, b in zip(got[:5], args))
    assert (got[5] is None) == (not start)
    for b in range(B):
        ref = od.delta_rule_backward(*(f64(t[b]) for t in args), 0.4, f64(dO[b]), f64(W0[b]) if start else None,
                                     f64(dWn[b]) if start else None)
        check([None if t is None else t[b] for t in got], ref, dtype, f"row {b}")


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("lens", [[70, 0, 5, 64, 129], [0, 0], [3], [64, 64, 64], [0, 200, 0]])
def test_packed_sequences(dtype, lens):
    Hk, Hv, dk, dv, front, behind = 1, 2, 64, 48, 5, 37
    n = front + sum(lens) + behind
    args = make(1, Hk, Hv, n, dk, dv, dtype, seed=len(lens))
    dO, _, _ = extras(1, Hv, n, dk, dv, dtype, "token")
    _, W0, dWn = extras(len(lens), Hv, 1, dk, dv, dtype, "token")
    for t in (*args, dO):
        t[:, :, :front] = float("nan")
        t[:, :, n - behind:] = float("nan")
    starts = torch.tensor([front] + lens).cumsum(0).to(torch.int32).cuda()
    outs = {x: torch.full_like(t, 7.0, dtype=dtype) for x, t in zip(NAMES, args)}
    got = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=W0, seq_starts=starts, **outs)
    for t in got[:5]:
        assert (t[:, :, :front] == 7).all() and (t[:, :, n - behind:] == 7).all()
    at = front
    for i, m in enumerate(lens):
        cut = lambda t: t[0, :, at:at + m]
        ref = od.delta_rule_backward(*(f64(cut(t)) for t in args), dk ** -0.5, f64(cut(dO)), f64(W0[i]), f64(dWn[i]))
        check([cut(t) for t in got[:5]] + [got[5][i]], ref, dtype, f"sequence {i} of {m}")
        at += m


@pytest.mark.parametrize("dtype", [F32, B16])
def test_resets_and_idle_tokens(dtype):
    args = make(1, 1, 2, 150, 64, 64, dtype, "head", seed=9)
    q, k, v, g, beta = args
    g[:, :, 64] = float("-inf")
    g[:, 0, 17] = float("-inf")
    g[:, 1, 100:] = -30.0
    beta[:, :, 20:30] = 0.0
    dO, _, _ = extras(1, 2, 150, 64, 64, dtype, "head")
    got = cw.ttt_gated_delta_backward(*args, dO)
    ref = od.delta_rule_backward(*(f64(t[0]) if t is not g else np.maximum(f64(t[0]), -700.0) for t in args), 64 ** -0.5,
                                 f64(dO[0]))
    check([None if t is None else t[0] for t in got], ref, dtype)
    # a gradient behind the reset does not reach what lies before it
    dO2 = torch.zeros_like(dO)
    dO2[:, :, 64:] = dO[:, :, 64:]
    for name, t in zip(NAMES[:3], cw.ttt_gated_delta_backward(*args, dO2)):
        assert not t[:, :, :64].any(), name


def test_differences():
    """Against central differences of the forward call itself (fp32; steps of 1e-2 leave O(1e-4) of curvature and
    2^-24 / 1e-2 of rounding in a sum of about 1e3: within 5e-3 of the largest)."""
    args = make(1, 1, 2, 90, 32, 40, F32, "head", seed=4)
    dO, W0, dWn = extras(1, 2, 90, 32, 40, F32, "head")
    args.append(W0)

    def loss(x):
        O, W = cw.ttt_gated_delta(*x[:5], W_init=x[5])
        return float((O.double() * dO.double()).sum() + (W.double() * dWn.double()).sum())

    got = cw.ttt_gated_delta_backward(*args[:5], dO, dW_final=dWn, W_init=W0)
    for i, d in enumerate(got):
        direction = torch.randn(d.shape, generator=torch.Generator().manual_seed(i)).cuda()
        direction /= direction.norm()
        ends = []
        for e in (1e-2, -1e-2):
            x = list(args)
            x[i] = args[i] + e * direction
            ends.append(loss(x))
        diff = (ends[0] - ends[1]) / 2e-2
        assert abs(diff - float((d.double() * direction.double()).sum())) <= 5e-3 * float(d.norm()), NAMES[i]


def test_repeated_gradient_and_same_bits():
    """dO repeated with stride 0 over tokens and heads (the gradient of a plain sum), at a length that ends inside a
    chunk; two calls give the same bits."""
    for dtype in (F32, B16):
        args = make(2, 1, 4, 100, 64, 64, dtype)
        dO = torch.ones(1, 1, 1, 64, dtype=dtype, device="cuda").expand(2, 4, 100, 64)
        a = cw.ttt_gated_delta_backward(*args, dO)
        b = cw.ttt_gated_delta_backward(*args, dO.contiguous())
        assert all(torch.equal(s, t) for s, t in zip(a[:5], b[:5]))


def test_empty_and_refusals():
    for B, n in ((0, 5), (2, 0)):
        args = make(B, 1, 2, n, 64, 64, B16, "head")
        W0 = torch.randn(B, 2, 64, 64, device="cuda")
        got = cw.ttt_gated_delta_backward(*args, torch.empty_like(args[2]), dW_final=W0, W_init=W0)
        assert got[0].shape == args[0].shape and torch.equal(got[5], W0)
    args = make(1, 1, 2, 40, 64, 64, B16, "head")
    dO, W0, dWn = extras(1, 2, 40, 64, 64, B16, "head")
    for err, change in ((TypeError, dict(dO=dO.float())), (ValueError, dict(dO=dO[:, :, :39])),
                        (ValueError, dict(dW_final=dWn[:, :1])), (TypeError, dict(dg=torch.empty(1, 2, 40, device="cuda"))),
                        (ValueError, dict(dv=dO[:, :1].expand(-1, 2, -1, -1))),
                        (ValueError, dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
                        (cw.TTTError, dict(scale=float("inf")))):
        with pytest.raises(err):
            cw.ttt_gated_delta_backward(*args, **(dict(dO=dO) | change))


def test_captured_replays_equal_the_eager_calls():
    """Captured while an eager autograd graph of the same leaves is alive."""
    args = make(2, 1, 2, 200, 128, 64, B16)
    dO, W0, dWn = extras(2, 2, 200, 128, 64, B16, "token")
    leaves = [t.requires_grad_() for t in args]
    alive = sum(t.float().sum() for t in leaves)
    call = lambda: cw.ttt_gated_delta_backward(*(t.detach() for t in leaves), dO, dW_final=dWn, W_init=W0)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        dO.mul_(1.5)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, call()):
            assert torch.equal(a, b)
    alive.backward()


@pytest.mark.parametrize("dtype", [F32, B16])
def test_rule_and_norm_of_its_heads_together(dtype):
    """A training step's run: the rule, a layer norm of each head's output, and both backward."""
    Hk, Hv, n, d = 2, 4, 140, 64
    args = make(1, Hk, Hv, n, d, d, dtype, "head")
    w = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(1))).to(dtype).cuda()
    dY, _, _ = extras(1, Hv, n, d, d, dtype, "head")
    O, _ = cw.ttt_gated_delta(*args)
    _, mean, rstd = cw.ttt_layer_norm(O, w)
    dO, dw, _ = cw.ttt_layer_norm_backward(O, w, dY, mean, rstd, bias=False)
    got = cw.ttt_gated_delta_backward(*args, dO)
    x = [f64(t[0]) for t in args]
    Or, _ = od.delta_rule(*x, d ** -0.5)
    _, mr, rr = od.layer_norm(Or.reshape(-1, d))
    dOr, dwr, _ = od.layer_norm_backward(Or.reshape(-1, d), f64(w), f64(dY).reshape(-1, d), mr, rr)
    ref = od.delta_rule_backward(*x, d ** -0.5, dOr.reshape(Or.shape))
    # O's roundings (2 2^-8, or 320 2^-24) go through the norm's gradient once more: added to each tolerance, twice
    # for rows of small spread
    extra = {B16: 8 * 2.0 ** -8, F32: 1280 * 2.0 ** -24}[dtype]
    for name, a, b in zip(NAMES + ("dw",), list(got[:5]) + [None, dw], list(ref[:5]) + [None, dwr]):
        if a is not None:
            a = f64(a).reshape(b.shape)
            assert np.linalg.norm(a - b) <= (TOL[dtype].get(name, 0.0) + extra) * np.linalg.norm(b), name
