"""The short causal convolution (forward, backward, single tokens) on the GPU against the oracle in fp64.

Tolerances (relative Frobenius norm).  fp32 sums of at most 9 terms, silu and its derivative from the hardware's
exponential and reciprocal, some 8 roundings of 2^-23 in all, whose errors stay below the norm of the terms: up to
2^-18 of the result where the taps' terms nearly cancel (random terms: their norm is at most 4 times the sum's).  bf16
outputs add a rounding of 2^-8.  The taps' and the bias's gradients: fp32 sums over the tokens, each thread's at most 64,
the runs' joined in a tree: 2^-17.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 2.0 ** -8 + 2.0 ** -18, torch.float32: 2.0 ** -18}
SUMS = 2.0 ** -17
DTYPES = [torch.float32, torch.bfloat16]


def rel(a, b):
    n = np.linalg.norm(b)
    a = a.double().cpu().numpy()
    return float(np.linalg.norm(a - b) / n) if n else float(np.abs(a).max(initial=0.0))


def f64(x):
    return None if x is None else x.double().cpu().numpy()


def make(B, n, d, K, rows, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype).cuda()
    return {"x": r(B, n, d), "w": r(d, K) / K ** 0.5, "bias": r(d), "x_init": r(rows, K - 1, d), "dY": r(B, n, d),
            "dx_final": r(rows, K - 1, d)}


CASES = [(1, 1, 8, 4), (2, 3, 16, 4), (1, 200, 72, 4), (3, 65, 13, 4), (1, 130, 2304, 4), (2, 40, 264, 1), (1, 33, 40, 2),
         (2, 50, 100, 3), (1, 64, 24, 5), (1, 97, 520, 8), (1, 5, 17, 8), (2, 31, 4104, 6), (1, 70, 48, 7)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("start", [False, True])
def test_forward_and_backward(case, dtype, start):
    B, n, d, K = case
    print("conv", case, dtype, start, flush=True)
    t = make(B, n, d, K, B, dtype)
    x0, dxf = (t["x_init"], t["dx_final"]) if start else (None, None)
    for bias, silu in ((t["bias"], True), (None, False)):
        Y, last = cw.ttt_short_conv(t["x"], t["w"], bias, silu=silu, x_init=x0)
        dx, dw, db, dx0 = cw.ttt_short_conv_backward(t["x"], t["w"], t["dY"], bias, silu=silu, x_init=x0, dx_final=dxf)
        assert (db is None) == (bias is None) and (dx0 is None) == (not start)
        dwr, dbr = 0, 0
        for b in range(B):
            args = [f64(v) for v in (t["x"][b], t["w"], bias)]
            i = f64(x0[b]) if start else None
            yr, lr = osc.short_conv(args[0], args[1], args[2], silu, i)
            assert rel(Y[b], yr) <= TOL[dtype] and np.array_equal(f64(last[b]), lr)
            g = osc.short_conv_backward(args[0], args[1], f64(t["dY"][b]), args[2], silu, i, f64(dxf[b]) if start else None)
            assert rel(dx[b], g[0]) <= TOL[dtype]
            assert not start or rel(dx0[b], g[3]) <= TOL[dtype]
            dwr, dbr = dwr + g[1], dbr + g[2]
        assert rel(dw, dwr) <= SUMS and (db is None or rel(db, dbr) <= SUMS)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [40, 19])
@pytest.mark.parametrize("lens", [[70, 0, 1, 64, 129], [0, 0], [3], [2, 2, 2, 1], [1] * 9, [0, 200, 0], []])
def test_packed_sequences(lens, d, dtype):
    """What lies in front of the first and behind the last sequence is not read (NaN) and stays as it was."""
    K, front, behind, num = 4, 5, 37, len(lens)
    n = front + sum(lens) + behind
    print("conv packed", lens, d, dtype, flush=True)
    t = make(1, n, d, K, num, dtype, seed=num)
    for v in (t["x"], t["dY"]):
        v[:, :front] = float("nan")
        v[:, n - behind:] = float("nan")
    starts = torch.tensor([front] + lens).cumsum(0).to(torch.int32).cuda()
    Y, dx = torch.full_like(t["x"], 7.0), torch.full_like(t["x"], 7.0)
    _, last = cw.ttt_short_conv(t["x"], t["w"], t["bias"], x_init=t["x_init"], seq_starts=starts, Y=Y)
    _, dw, db, dx0 = cw.ttt_short_conv_backward(t["x"], t["w"], t["dY"], t["bias"], x_init=t["x_init"], seq_starts=starts,
                                                dx_final=t["dx_final"], dx=dx)
    for v in (Y, dx):
        assert (v[:, :front] == 7).all() and (v[:, n - behind:] == 7).all()
    at, dwr, dbr = front, np.zeros((d, K)), np.zeros(d)
    for i, m in enumerate(lens):
        x, dy = f64(t["x"][0, at:at + m]), f64(t["dY"][0, at:at + m])
        yr, lr = osc.short_conv(x, f64(t["w"]), f64(t["bias"]), True, f64(t["x_init"][i]))
        g = osc.short_conv_backward(x, f64(t["w"]), dy, f64(t["bias"]), True, f64(t["x_init"][i]), f64(t["dx_final"][i]))
        assert rel(Y[0, at:at + m], yr) <= TOL[dtype] and np.array_equal(f64(last[i]), lr), (i, m)
        assert rel(dx[0, at:at + m], g[0]) <= TOL[dtype] and rel(dx0[i], g[3]) <= TOL[dtype], (i, m)
        dwr, dbr, at = dwr + g[1], dbr + g[2], at + m
    assert rel(dw, dwr) <= SUMS and rel(db, dbr) <= SUMS


def test_starts_outside_the_row_do_not_lead_out_of_it():
    t = make(1, 50, 16, 4, 3, torch.float32)
    starts = torch.tensor([-7, 20, 1 << 30, 1 << 30], dtype=torch.int32, device="cuda")
    Y, last = cw.ttt_short_conv(t["x"], t["w"], x_init=t["x_init"], seq_starts=starts)
    ref = cw.ttt_short_conv(t["x"], t["w"], x_init=t["x_init"],
                            seq_starts=torch.tensor([0, 20, 50, 50], dtype=torch.int32, device="cuda"))
    assert torch.equal(Y, ref[0]) and torch.equal(last, ref[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides(dtype):
    """Slices of a wider projection, whole vectors and not, token-major and batch-major."""
    t = make(2, 40, 64, 4, 2, dtype)
    ref = cw.ttt_short_conv(t["x"], t["w"], t["bias"])
    back = cw.ttt_short_conv_backward(t["x"], t["w"], t["dY"], t["bias"])
    for off, width in ((16, 128), (3, 71)):
        wide = torch.zeros(40, 2, width, dtype=dtype, device="cuda")
        x = wide[:, :, off:off + 64].transpose(0, 1).copy_(t["x"])
        Y = torch.zeros(40, 2, width, dtype=dtype, device="cuda")[:, :, off:off + 64].transpose(0, 1)
        out, last = cw.ttt_short_conv(x, t["w"], t["bias"], Y=Y)
        assert out is Y and torch.equal(Y, ref[0]) and torch.equal(last, ref[1])
        dY = torch.zeros_like(wide)[:, :, off:off + 64].transpose(0, 1).copy_(t["dY"])
        dx = torch.zeros_like(wide)[:, :, off:off + 64].transpose(0, 1)
        got = cw.ttt_short_conv_backward(x, t["w"], dY, t["bias"], dx=dx)
        assert torch.equal(dx, back[0]) and torch.equal(got[1], back[1]) and torch.equal(got[2], back[2])
    # one row for all tokens
    same = t["x"][:, :1].expand(2, 40, 64)
    assert torch.equal(cw.ttt_short_conv(same, t["w"])[0], cw.ttt_short_conv(same.contiguous(), t["w"])[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [(1, 2, 8, 4), (9, 12, 72, 4), (5, 5, 13, 4), (4, 7, 2304, 2), (3, 4, 24, 1), (6, 8, 100, 8)])
def test_step(case, dtype):
    R, P, d, K = case
    print("conv step", case, dtype, flush=True)
    t = make(1, R, d, K, P, dtype, 3)
    slots = torch.randperm(P, generator=torch.Generator().manual_seed(1))[:R].to(torch.int32).cuda()
    if R > 2:
        slots[1], slots[-1] = -1, P
    for named in (True, False):
        halo = t["x_init"].clone()
        Y = cw.ttt_short_conv_step(t["x"][0], t["w"], halo, t["bias"], slots=slots if named else None)
        want = t["x_init"].clone()
        for r in range(R):
            s = int(slots[r]) if named else r
            if not 0 <= s < P:
                assert (Y[r] == 0).all()
                continue
            yr, lr = osc.short_conv(f64(t["x"][0, r:r + 1]), f64(t["w"]), f64(t["bias"]), True, f64(t["x_init"][s]))
            assert rel(Y[r:r + 1], yr) <= TOL[dtype]
            want[s] = torch.tensor(lr).to(dtype)
        assert torch.equal(halo, want)


@pytest.mark.parametrize("d", [64, 33])
def test_rows_of_one_slot_go_in_row_order(d):
    """Tokens of one sequence given as rows of one call: as if they came one call after another, or as a sequence."""
    t = make(1, 700, d, 4, 3, torch.float32)
    order = torch.randint(0, 3, (700,), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    halo = t["x_init"].clone()
    Y = cw.ttt_short_conv_step(t["x"][0], t["w"], halo, slots=order)
    for s in range(3):
        mine = (order == s).nonzero()[:, 0]
        ref, last = cw.ttt_short_conv(t["x"][:, mine], t["w"], x_init=t["x_init"][s:s + 1])
        assert torch.equal(Y[mine], ref[0]) and torch.equal(halo[s:s + 1], last)


def test_prompt_then_tokens_is_the_sequence():
    t = make(2, 30, 48, 4, 2, torch.bfloat16)
    Y, last = cw.ttt_short_conv(t["x"], t["w"], t["bias"])
    head, halo = cw.ttt_short_conv(t["x"][:, :20], t["w"], t["bias"])
    assert torch.equal(head, Y[:, :20])
    for i in range(20, 30):
        y = cw.ttt_short_conv_step(t["x"][:, i].contiguous(), t["w"], halo, t["bias"])
        assert torch.equal(y, Y[:, i])
    assert torch.equal(halo, last)


def test_refusals():
    t = make(2, 30, 48, 4, 2, torch.bfloat16)
    x, w = t["x"], t["w"]
    for bad in (dict(conv_w=w.float()), dict(conv_w=w[:40]), dict(bias=t["bias"][:40]), dict(x_init=t["x_init"][:1]),
                dict(seq_starts=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(Y=x[:1].expand(2, 30, 48)),
                dict(Y=x[:, :20]), dict(x=x.transpose(1, 2)), dict(x=x.cpu()), dict(x=x.half())):
        with pytest.raises((ValueError, TypeError)):
            cw.ttt_short_conv(**{"x": x, "conv_w": w, **bad})
    with pytest.raises(cw.TTTError):
        cw.ttt_short_conv(x, torch.zeros(48, 9, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        cw.ttt_short_conv_backward(x, w, t["dY"][:, :20])
    with pytest.raises(ValueError):
        cw.ttt_short_conv_step(x[0], w, t["x_init"][:, :2])
    with pytest.raises(cw.TTTError):
        cw.ttt_short_conv_step(x[0], w, t["x_init"])         # more rows than states
