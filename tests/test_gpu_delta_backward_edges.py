"""The gated delta rule's backward at the edges of what it takes.  Tolerances are those of test_gpu_delta_backward."""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import delta as od
from test_gpu_delta import TOL_O, TOL_W, f64, make, rel
from test_gpu_delta_backward import B16, F32, NAMES, TOL, extras

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("n", [64, 128, 257])
def test_no_sequences(dtype, n):
    """A single start, the first entry of a longer tensor whose next one is the row's length: every gradient's rows stay
    as they are."""
    args = make(1, 1, 2, n, 64, 64, dtype, "head")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")[:1]
    outs = {x: torch.full_like(t, 7.0, dtype=dtype) for x, t in zip(NAMES, args)}
    got = cw.ttt_gated_delta_backward(*args, torch.ones_like(args[2]), seq_starts=starts, **outs)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in got[:5]) and got[5] is None


@pytest.mark.parametrize("dtype", [F32, B16])
def test_small_gradients_of_strong_decays(dtype):
    """dg_t is of the size of exp(g_t): it keeps its digits, head by head, under decays that are strong throughout (-8,
    -12, -16) and, token by token, under single ones of -14 among weak ones, inside a chunk and at its ends, where the
    neighbours' gradients are larger by a factor of 10^6.  (exp's own error at -16 is 2 * 16 * 2^-24, 2e-6.)"""
    Hv, n = 4, 200
    args = make(1, 2, Hv, n, 32, 40, dtype, "head", seed=11)
    dO, W0, dWn = extras(1, Hv, n, 32, 40, dtype, "head")
    g = args[3]
    for h, x in enumerate((-8.0, -12.0, -16.0)):
        g[:, h] = x
    g[:, 3] = -0.02
    strong = [5, 31, 32, 40, 63, 64, 100, 127, 128, 150, 191, 192, 199]
    g[:, 3, strong] = -14.0
    got = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=W0)
    ref = od.delta_rule_backward(*(f64(t[0]) for t in args), 32 ** -0.5, f64(dO[0]), f64(W0[0]), f64(dWn[0]))
    dg, want = f64(got[3][0]), ref[3]
    weak = [t for t in range(n) if t not in strong]
    parts = [(0, slice(None)), (1, slice(None)), (2, slice(None)), (3, strong), (3, weak)]
    errs = [np.linalg.norm(dg[h, at] - want[h, at]) / np.linalg.norm(want[h, at]) for h, at in parts]
    print(dtype, errs, flush=True)
    assert max(errs) <= TOL[dtype]["dg"], errs
    for name, a, b in zip(NAMES, got, ref):
        for h in range(Hv if b.shape[0] == Hv else 0):
            e = np.linalg.norm(f64(a[0, h]) - b[h]) / np.linalg.norm(b[h])
            assert e <= TOL[dtype][name], (name, h, e)


def test_gradient_of_a_reset_is_zero():
    """A decay of zero (g = -inf): nothing passes it, and dg there is zero itself, not what a cancelled sum leaves."""
    for dtype in (F32, B16):
        args = make(1, 1, 2, 150, 64, 64, dtype, "head", seed=9)
        at = [0, 17, 64, 127, 149]
        args[3][:, :, at] = float("-inf")
        dO, W0, dWn = extras(1, 2, 150, 64, 64, dtype, "head")
        dg = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=W0)[3]
        assert not dg[:, :, at].any() and not dg.isnan().any()


@pytest.mark.parametrize("layout", ["head", "token"])
def test_gate_gradients_in_fp32(layout):
    """g and beta are fp32, and so are their gradients where asked for: the same sums, not rounded to the inputs' type."""
    args = make(2, 2, 4, 130, 64, 72, B16, layout, seed=21)
    dO, W0, dWn = extras(2, 4, 130, 64, 72, B16, layout)
    call = lambda **o: cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=W0, **o)
    low, full = call(), call(gate_dtype=F32)
    assert full[3].dtype == full[4].dtype == F32 and full[3].stride() == args[3].stride()
    assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(low, full)) if i not in (3, 4))
    for i in (3, 4):
        assert torch.equal(full[i].to(B16), low[i]) and not torch.equal(full[i], low[i].float())
    out = torch.full((2, 130, 5, 4), 7.0, device="cuda")                    # given, between other values
    given = [out[:, :, i].transpose(1, 2) for i in (1, 3)]
    call(gate_dtype=F32, dg=given[0], dbeta=given[1])
    assert torch.equal(given[0], full[3]) and torch.equal(given[1], full[4]) and (out[:, :, ::2] == 7).all()
    assert call(gate_dtype=B16)[3].dtype == B16
    for err, o in ((TypeError, dict(gate_dtype=torch.float16)), (TypeError, dict(gate_dtype=F32, dg=low[3])),
                   (TypeError, dict(gate_dtype=B16, dbeta=full[4]))):
        with pytest.raises(err):
            call(**o)
    x = make(1, 1, 1, 5, 64, 64, F32)
    assert cw.ttt_gated_delta_backward(*x, torch.ones_like(x[2]))[3].dtype == F32
    with pytest.raises(TypeError):
        cw.ttt_gated_delta_backward(*x, torch.ones_like(x[2]), gate_dtype=B16)


def check_by_scale(got, ref, dtype, what):
    """As test_gpu_delta_backward's check, with an error measured against the largest gradient's norm where a gradient is
    zero in exact arithmetic (dg and parts of dk of a sequence's first tokens)."""
    largest = max(float(np.abs(b).max(initial=0.0)) for b in ref)
    for name, a, b in zip(NAMES, got, ref):
        if a is None:
            continue
        n = np.linalg.norm(b)
        err = np.linalg.norm(f64(a) - b) / (n if n > 1e-12 else largest * b.size ** 0.5)
        print("  ", what, name, err, flush=True)
        assert err <= TOL[dtype][name], (what, name)


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("start", [False, True])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 72), (256, 128)])
def test_one_and_two_tokens(dk, dv, start, n, dtype):
    B, Hk, Hv = 3, 2, 4
    args = make(B, Hk, Hv, n, dk, dv, dtype, seed=41)
    dO, W0, dWn = extras(B, Hv, n, dk, dv, dtype, "token")
    if not start:
        W0 = dWn = None
    got = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=W0)
    refs = [od.delta_rule_backward(*(f64(t[b]) for t in args), dk ** -0.5, f64(dO[b]), f64(W0[b]) if start else None,
                                   f64(dWn[b]) if start else None) for b in range(B)]
    ref = [np.stack(r) for r in zip(*refs)]
    check_by_scale(got if start else got[:5], ref, dtype, f"{n} tokens")


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("lens", [[70, 0, 1, 64, 129], [1] * 9, [2, 1, 1, 0, 2, 65, 1]])
def test_packed_single_tokens(lens, dtype):
    """All sequences' gradients of a kind together: a gate's gradient of one token is one number, whose own error has no
    norm to be held against."""
    Hk, Hv, dk, dv, front, behind = 1, 2, 64, 48, 5, 37
    n = front + sum(lens) + behind
    args = make(1, Hk, Hv, n, dk, dv, dtype, seed=len(lens))
    dO, _, _ = extras(1, Hv, n, dk, dv, dtype, "token")
    _, W0, dWn = extras(len(lens), Hv, 1, dk, dv, dtype, "token")
    for t in (*args, dO):
        t[:, :, :front] = float("nan")
        t[:, :, n - behind:] = float("nan")
    starts = torch.tensor([front] + lens).cumsum(0).to(torch.int32)
    outs = {x: torch.full_like(t, 7.0, dtype=dtype) for x, t in zip(NAMES, args)}
    got = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=W0, seq_starts=starts.cuda(), **outs)
    refs = []
    for i, m in enumerate(lens):
        cut = lambda t: f64(t[0, :, int(starts[i]):int(starts[i]) + m])
        refs.append(od.delta_rule_backward(*(cut(t) for t in args), dk ** -0.5, cut(dO), f64(W0[i]), f64(dWn[i])))
    ref = [np.concatenate(r, 1) for r in list(zip(*refs))[:5]] + [np.stack([r[5] for r in refs])]
    for t in got[:5]:
        assert (t[:, :, :front] == 7).all() and (t[:, :, n - behind:] == 7).all()
    check_by_scale([t[0, :, front:n - behind] for t in got[:5]] + [got[5]], ref, dtype, f"{lens}")


@pytest.mark.parametrize("dtype", [F32, B16])
def test_reset_at_the_first_token_clears_any_state(dtype):
    """As in the forward pass: the state to start from is not looked at, and its gradient is zero."""
    args = make(2, 1, 2, 100, 64, 48, dtype, "head", seed=51)
    dO, W0, dWn = extras(2, 2, 100, 64, 48, dtype, "head")
    args[3][1, :, 0] = float("-inf")
    zero = W0.clone()
    W0[1], zero[1] = float("nan"), 0.0
    got = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=W0)
    ref = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=zero)
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and not got[5][1].any() and got[5][0].any()


@pytest.mark.parametrize("dtype", [F32, B16])
def test_values_that_are_not_finite_stay_in_their_sequence_and_key_heads(dtype):
    lens, Hk, Hv = [70, 64, 100, 5], 2, 4
    n = sum(lens)
    args = make(1, Hk, Hv, n, 64, 64, dtype, seed=53)
    dO = extras(1, Hv, n, 64, 64, dtype, "token")[0]
    starts = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    call = lambda x, d: cw.ttt_gated_delta_backward(*x, d, seq_starts=starts.cuda())
    ref = call(args, dO)
    inside = torch.zeros(n, dtype=torch.bool, device="cuda")
    inside[int(starts[1]):int(starts[2])] = True
    for t in range(6):                                                     # dO is the last
        bad = [x.clone() for x in (*args, dO)]
        bad[t][:, 0, 75] = float("nan")
        got = call(bad[:5], bad[5])
        for a, b in zip(got[:5], ref):
            other = slice(1, None) if a.shape[1] == Hk else slice(Hv // Hk, None)
            assert torch.equal(a[:, other], b[:, other]) and torch.equal(a[:, :, ~inside], b[:, :, ~inside])


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("dk,dv", [(64, 4096), (256, 520), (8, 8), (192, 104), (136, 264)])
def test_widths_between_and_at_the_limits(dk, dv, dtype):
    """Forward and backward of the widest values, of keys between the kernels' widths, and of the narrowest heads."""
    args = make(1, 1, 2, 70, dk, dv, dtype, seed=61)
    dO, W0, dWn = extras(1, 2, 70, dk, dv, dtype, "token")
    O, W = cw.ttt_gated_delta(*args, W_init=W0)
    got = cw.ttt_gated_delta_backward(*args, dO, dW_final=dWn, W_init=W0)
    x = [f64(t[0]) for t in args]
    Or, Wr = od.delta_rule(*x, dk ** -0.5, f64(W0[0]))
    assert rel(O[0], Or) <= TOL_O[dtype] and rel(W[0], Wr) <= TOL_W[dtype]
    ref = od.delta_rule_backward(*x, dk ** -0.5, f64(dO[0]), f64(W0[0]), f64(dWn[0]))
    check_by_scale([t[0] for t in got], ref, dtype, f"{dk} x {dv}")


@pytest.mark.parametrize("dtype", [F32, B16])
def test_largest_token_strides(dtype):
    """Tokens 2^22 elements apart, the most that is taken, one tensor at a time, given and written."""
    n, d, far = 70, 64, 1 << 22
    args = make(1, 1, 1, n, d, d, dtype, "head", seed=62)
    dO = extras(1, 1, n, d, d, dtype, "head")[0]
    base = torch.empty((n - 1) * far + d, dtype=dtype, device="cuda")
    wide = base.as_strided((1, 1, n, d), (n * far, far, far, 1))
    ref, grads = cw.ttt_gated_delta(*args), cw.ttt_gated_delta_backward(*args, dO)
    for i in range(4):
        x = [*args[:3], dO]
        wide.copy_(x[i])
        x[i] = wide
        got = cw.ttt_gated_delta(*x[:3], *args[3:])
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        assert all(torch.equal(a, b) for a, b in zip(cw.ttt_gated_delta_backward(*x[:3], *args[3:], x[3]), grads[:5]))
    assert torch.equal(cw.ttt_gated_delta(*args, O=wide)[0], ref[0])
    for i, name in enumerate(NAMES[:3]):
        wide.zero_()
        assert torch.equal(cw.ttt_gated_delta_backward(*args, dO, **{name: wide})[i], grads[i])
    with pytest.raises(cw.TTTError):
        cw.ttt_gated_delta(base.as_strided((1, 1, 3, d), (3 * far, far, far + 64, 1)), *(t[:, :, :3] for t in args[1:]))
