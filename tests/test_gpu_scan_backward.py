"""Backward of the selective scan on the GPU against the oracle's reverse recurrence in fp64, and against differences.

Tolerances (relative Frobenius norm).  A rounding to bf16 is off by at most half a step, 2^-8 of the value; fp32 by 2^-24.
  bf16 inputs   states, their gradients, decayed products and weights enter products as pairs of bf16 values, 2^-16 off:
                four of them one behind the other in a term, 2^-14, and a gradient of terms whose norm is at most 8 times
                its own in these random inputs: 2^-11.  dx, dB and dC add their own rounding, 2^-8.
  dA, dD, ddt_bias are sums of the sequences' own: their errors are relative to those, not to a sum in which they cancel
                (sequences' dA of some 1400 in three rows of one head add up to -0.9, off by 0.0035: 2.5e-6 of them).
  fp32 inputs   sums of at most 320 terms, twice one behind the other, of terms of the same spread: 8 * 640 * 2^-24 = 2^-11.7.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc
from tests.test_gpu_scan import CASES, DTYPES, f64, make, rel

pytestmark = pytest.mark.gpu

SUMS = {torch.bfloat16: 2.0 ** -11, torch.float32: 8 * 640 * 2.0 ** -24}
OUT = {torch.bfloat16: 2.0 ** -8 + 2.0 ** -11, torch.float32: 8 * 640 * 2.0 ** -24}
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dS0")


def tol(name, dtype):
    return (OUT if name in ("dx", "dB", "dC") else SUMS)[dtype]


def reference(args, dO, D, bias, softplus, S0, dS, parts):
    """The oracle's gradients of several sequences (batch row, tokens), those of the vectors summed."""
    x, dt, A, B, C = args
    out, total = [], {}
    for i, (b, cut) in enumerate(parts):
        one = [f64(v[b][:, cut]) if v.dim() > 1 else f64(v) for v in args]
        d = osc.selective_scan_backward(*one, f64(dO[b][:, cut]), f64(D), f64(bias), softplus,
                                        None if S0 is None else f64(S0[i]), None if dS is None else f64(dS[i]))
        out.append(d)
        for n in ("dA", "dD", "ddt_bias"):
            total[n] = total.get(n, 0) + d[n]
    return out, total


def check(grads, ref, total, parts, dtype, S0, D, bias):
    got = dict(zip(NAMES, grads))
    for i, (b, cut) in enumerate(parts):
        for n in ("dx", "ddt", "dB", "dC"):
            assert rel(got[n][b][:, cut], ref[i][n]) <= tol(n, dtype), (n, i, rel(got[n][b][:, cut], ref[i][n]))
        if S0 is not None:
            assert rel(got["dS0"][i], ref[i]["dS0"]) <= tol("dS0", dtype), ("dS0", i)
    for n, there in (("dA", True), ("dD", D is not None), ("ddt_bias", bias is not None)):
        assert (got[n] is not None) == there
        if there:
            size = np.sqrt(sum(np.linalg.norm(d[n]) ** 2 for d in ref))
            off = np.linalg.norm(f64(got[n]) - total[n])
            assert off <= tol(n, dtype) * size, (n, off, size)
    assert (got["dS0"] is not None) == (S0 is not None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("start", [False, True])
def test_sequence(case, dtype, start):
    B, H, G, n, P, N, layout = case
    print("scan backward", case, dtype, start, flush=True)
    *args, D, bias = make(B, H, G, n, P, N, dtype, layout, seed=1)
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    dO = r(B, n, H, P).to(dtype).transpose(1, 2)
    S0, dS = (r(B, H, P, N) * 0.3, r(B, H, P, N)) if start else (None, None)
    D, bias = (D, bias) if start else (None, None)
    grads = cw.ttt_selective_scan_backward(*args, dO, D=D, dt_bias=bias, softplus=True, dS_final=dS, S_init=S0)
    parts = [(b, slice(None)) for b in range(B)]
    ref, total = reference(args, dO, D, bias, True, S0, dS, parts)
    check(grads, ref, total, parts, dtype, S0, D, bias)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[70, 0, 1, 64, 129], [0, 0], [3], [1] * 9, [0, 700, 0], [300, 257, 0, 256, 513], []])
def test_packed_sequences(dtype, lens):
    H, G, P, N, front, behind = 4, 2, 48, 64, 5, 37
    n, num = front + sum(lens) + behind, len(lens)
    print("scan backward packed", lens, dtype, flush=True)
    *args, D, bias = make(1, H, G, n, P, N, dtype, seed=num)
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    dO = r(1, n, H, P).to(dtype).transpose(1, 2)
    for t in (args[0], args[1], args[3], args[4], dO):
        t[:, :, :front] = float("nan")
        t[:, :, n - behind:] = float("nan")
    starts = torch.tensor([front] + lens).cumsum(0).to(torch.int32).cuda()
    S0, dS = r(num, H, P, N) * 0.3, r(num, H, P, N)
    outs = [torch.full_like(t, 7.0) for t in (args[0], args[1], args[3], args[4])]
    grads = cw.ttt_selective_scan_backward(*args, dO, D=D, dt_bias=bias, softplus=True, dS_final=dS, S_init=S0,
                                           seq_starts=starts, dx=outs[0], ddt=outs[1], dB=outs[2], dC=outs[3])
    for o in outs:
        assert (o[:, :, :front] == 7).all() and (o[:, :, n - behind:] == 7).all()
    parts, at = [], front
    for m in lens:
        parts.append((0, slice(at, at + m)))
        at += m
    ref, total = reference(args, dO, D, bias, True, S0, dS, parts)
    if not lens:
        total = {n: np.zeros(H) for n in ("dA", "dD", "ddt_bias")}
    check(grads, ref, total, parts, dtype, S0, D, bias)
    for i, m in enumerate(lens):
        if m == 0:
            assert torch.equal(grads[7][i], dS[i])


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_softplus_idle_tokens_and_emptied_states(dtype):
    x, dt, A, B, C, D, _ = make(1, 2, 1, 500, 64, 64, dtype, "head", seed=9)
    dt = dt.abs() * 0.3
    dt[:, :, 20:30] = 0.0
    dt[:, :, 64:70] = 0.0
    dt[:, 1, 140:170] = 20.0
    dt[:, :, 300] = 1e4
    dt[:, 0, 17] = 1e4
    A[:] = torch.tensor([-1.0, -2.0])
    dO = torch.randn(1, 2, 500, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    grads = cw.ttt_selective_scan_backward(x, dt, A, B, C, dO, D=D)
    ref, total = reference((x, dt, A, B, C), dO, D, None, False, None, None, [(0, slice(None))])
    # tokens of rate 1e4 have gradients that size: each kind of token by itself
    big = torch.zeros(500, dtype=torch.bool)
    big[[17, 300]] = True
    for n, g in zip(NAMES, grads):
        if n in ("dx", "ddt", "dB", "dC"):
            for sel in (big, ~big):
                assert rel(g[0][:, sel.cuda()], ref[0][n][:, sel.numpy()]) <= tol(n, dtype), n


@pytest.mark.parametrize("dtype", DTYPES)
def test_along_directions_against_differences(dtype):
    """<gradient, direction> against central differences of the oracle's loss, whose own error is some 1e-7."""
    *args, D, bias = make(1, 4, 2, 90, 32, 24, dtype, "head", seed=6)
    gen = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    dO, S0, dS = r(1, 4, 90, 32).to(dtype), r(1, 4, 32, 24), r(1, 4, 32, 24)
    grads = cw.ttt_selective_scan_backward(*args, dO, D=D, dt_bias=bias, softplus=True, dS_final=dS, S_init=S0)
    vals = [f64(v[0]) if v.dim() > 1 else f64(v) for v in (*args, D, bias, S0)]
    order = (0, 1, 2, 3, 4, 5, 6, 7)

    def loss(v):
        O, S = osc.selective_scan(*v[:7], True, v[7])
        return (O * f64(dO[0])).sum() + (S * f64(dS[0])).sum()

    rng = np.random.default_rng(0)
    for i, (n, g) in enumerate(zip(NAMES, grads)):
        g = f64(g[0]) if g.dim() > 1 else f64(g)
        step = rng.normal(size=vals[i].shape) + 3 * np.sign(g)     # towards the gradient, so that the product is large
        move = lambda e: [v + e * step if k == i else v for k, v in enumerate(vals)]
        diff = (loss(move(1e-6)) - loss(move(-1e-6))) / 2e-6
        assert abs((g * step).sum() - diff) <= tol(n, dtype) * np.linalg.norm(g) * np.linalg.norm(step) + 1e-6 * abs(diff), n


@pytest.mark.parametrize("dtype", DTYPES)
def test_shared_groups_and_zero_strides(dtype):
    """B and C of one group repeated over the heads by zero strides: their gradients' sums are the group's."""
    x, dt, A, B, C, D, bias = make(2, 4, 1, 130, 64, 32, dtype, "head")
    dO = torch.randn(2, 4, 130, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    kw = dict(D=D, dt_bias=bias, softplus=True)
    one = cw.ttt_selective_scan_backward(x, dt, A, B, C, dO, **kw)
    each = cw.ttt_selective_scan_backward(x, dt, A, B.expand(2, 4, 130, 32), C.expand(2, 4, 130, 32), dO,
                                          dB=torch.empty(2, 4, 130, 32, dtype=dtype, device="cuda"),
                                          dC=torch.empty(2, 4, 130, 32, dtype=dtype, device="cuda"), **kw)
    for i in (3, 4):
        assert rel(one[i][:, 0].float(), f64(each[i].float().sum(1))) <= 2 * OUT[dtype]
    for i in (0, 1, 2, 5, 6):
        assert rel(one[i], f64(each[i])) <= 2 * tol(NAMES[i], dtype)


def test_refusals():
    x, dt, A, B, C, D, bias = make(2, 4, 2, 50, 64, 32, torch.bfloat16, "head")
    good = dict(x=x, dt=dt, A=A, B=B, C=C, dO=x)
    for bad in (dict(dO=x.float()), dict(dO=x[:, :, :20]), dict(dx=x[:, :1].expand(2, 4, 50, 64)), dict(ddt=dt.bfloat16()),
                dict(dA=A[:2]), dict(dD=A.bfloat16()), dict(dS_final=torch.zeros(2, 4, 64, 16, device="cuda")),
                dict(dB=B.float()), dict(workspace=torch.empty(0, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            cw.ttt_selective_scan_backward(**{**good, **bad})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sums_over_tokens_of_fast_heads(dtype):
    """Heads that forget within a few tokens: dA and ddt_bias are sums over thousands of tokens of either sign.  A token's
    part is off by at most 16 roundings (2^-24) of its own size, each by itself, and the exact sum has the size of as many
    parts of random sign: 16 * 2^-24 of it.  What errors of a token passed on to those behind it came to was four times
    that and more."""
    H, n = 8, 2048
    *args, D, _ = make(1, H, 1, n, 64, 128, dtype, seed=9)
    args[2] = torch.linspace(-16, -12, H).cuda()
    bias = torch.full((H,), -2.25, device="cuda")
    dO = torch.randn(args[0].shape, generator=torch.Generator().manual_seed(10)).to(dtype).cuda()
    got = cw.ttt_selective_scan_backward(*args, dO, D=D, dt_bias=bias, softplus=True)
    want = osc.selective_scan_backward(*(f64(t[0]) if t.dim() > 1 else f64(t) for t in args), f64(dO[0]), f64(D), f64(bias), True)
    for t, k in ((got[2], "dA"), (got[6], "ddt_bias")):
        print(k, rel(t, want[k]), flush=True)
        assert rel(t, want[k]) <= 16 * 2.0 ** -24, k
