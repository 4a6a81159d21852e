"""Layer norm, forward and backward, on the GPU against the oracle in fp64.

Tolerances (relative Frobenius norm): fp32 sums of up to 2^16 terms, kept by each thread over at most 64 and joined in
a tree, 2^7 roundings of 2^-24 deep: 2^-17 at most; bf16 outputs add one rounding, 2^-8.
The weight's and the bias's gradient: fp32 sums over the rows, each thread's at most 64 in the tests' sizes and joined
the same way: 2^-17.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
import ttt_inputs as ti
from oracle import delta as od
from oracle import inplace as orc

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 2.0 ** -8 + 2.0 ** -17, torch.float32: 2.0 ** -17}
SUM_TOL = 2.0 ** -17
DTYPES = [torch.float32, torch.bfloat16]


def rel(a, b):
    n = np.linalg.norm(b)
    a = a.double().cpu().numpy()
    return float(np.linalg.norm(a - b) / n) if n else float(np.abs(a).max(initial=0.0))


def f64(x):
    return None if x is None else x.double().cpu().numpy()


# rows and widths of every variant: parts of a wave, waves, workgroups of 256 and 1024; whole vectors and not
SIZES = [(1, 8), (5, 128), (1, 1), (37, 100), (3, 512), (9, 1001), (4, 1536), (6, 2560), (300, 264), (2, 4096), (3, 5000),
         (2, 8192), (2, 9001), (1, 16384), (2, 20000), (1, 65536), (1, 40001), (2000, 72)]


def make(rows, d, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    x = (r(rows, d) * (0.5 + torch.rand(rows, 1, generator=gen)) + r(rows, 1)).to(dtype).cuda()
    return x, (1 + 0.3 * r(d)).to(dtype).cuda(), r(d).to(dtype).cuda(), r(rows, d).to(dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", SIZES)
def test_forward_and_backward(size, dtype):
    rows, d = size
    print("norm", size, dtype, flush=True)
    x, w, b, dy = make(rows, d, dtype)
    for weight, bias in ((w, b), (w, None), (None, b), (None, None)):
        y, mean, rstd = cw.ttt_layer_norm(x, weight, bias, eps=1e-4)
        yr, mr, rr = od.layer_norm(f64(x), f64(weight), f64(bias), 1e-4)
        assert rel(y, yr) <= TOL[dtype] and rel(mean, mr) <= 2.0 ** -17 and rel(rstd, rr) <= 2.0 ** -17
        dx, dw, db = cw.ttt_layer_norm_backward(x, weight, dy, mean, rstd, bias=bias is not None)
        dxr, dwr, dbr = od.layer_norm_backward(f64(x), f64(weight), f64(dy), f64(mean), f64(rstd))
        if d > 2:                 # a row of one or two: dx is zero but for roundings
            assert rel(dx, dxr) <= TOL[dtype]
        assert (dw is None) == (weight is None) and (db is None) == (bias is None)
        assert dw is None or rel(dw, dwr) <= SUM_TOL
        assert db is None or rel(db, dbr) <= SUM_TOL


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_offset_keeps_its_digits(dtype):
    """Rows far from zero: the variance is taken around the mean, not from the squares' mean.  The offset (1024) is
    exact in both types; fp32 rounds the mean by 2^-24 * 1024, 6e-5 of the spread 1, and every other step by less."""
    x = (1024 + 8 * torch.randint(-3, 4, (7, 1000), generator=torch.Generator().manual_seed(2))).to(dtype).cuda()
    y, mean, rstd = cw.ttt_layer_norm(x)
    yr, _, _ = od.layer_norm(f64(x))
    assert rel(y, yr) <= TOL[dtype] + 1024 * 2.0 ** -24


def test_rows_with_infinities_stay_alone():
    x, w, b, dy = make(9, 256, torch.float32)
    ref = cw.ttt_layer_norm(x, w, b)[0]
    x2 = x.clone()
    x2[3, 7] = float("inf")
    x2[5, 1] = float("nan")
    y = cw.ttt_layer_norm(x2, w, b)[0]
    keep = [i for i in range(9) if i not in (3, 5)]
    assert torch.equal(y[keep], ref[keep]) and y[3].isnan().any() and y[5].isnan().all()


def test_empty_and_shapes():
    w = torch.ones(64, device="cuda")
    y, mean, rstd = cw.ttt_layer_norm(torch.empty(0, 64, device="cuda"), w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = cw.ttt_layer_norm_backward(torch.empty(0, 64, device="cuda"), w, torch.empty(0, 64, device="cuda"), mean,
                                            rstd)
    assert not dw.any() and not db.any()
    x = torch.randn(2, 3, 5, 64, device="cuda")
    y, mean, rstd = cw.ttt_layer_norm(x, w)
    assert y.shape == x.shape and mean.shape == (2, 3, 5)


def test_many_rows_and_the_same_bits_each_time():
    x, w, b, dy = make(70001, 128, torch.bfloat16)
    y, mean, rstd = cw.ttt_layer_norm(x, w, b)
    first = cw.ttt_layer_norm_backward(x, w, dy, mean, rstd)
    again = cw.ttt_layer_norm_backward(x, w, dy, mean, rstd)
    assert all(torch.equal(s, t) for s, t in zip(first, again))
    ref = od.layer_norm_backward(f64(x), f64(w), f64(dy), f64(mean), f64(rstd))
    # each thread sums 70001 / 4096 / 4 rows: the bound above holds
    for a, r, tol in zip(first, ref, (TOL[torch.bfloat16], SUM_TOL, SUM_TOL)):
        assert rel(a, r) <= tol


def test_refusals():
    x, w, b, dy = make(4, 64, torch.float32)
    mean, rstd = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
    for err, call in ((TypeError, lambda: cw.ttt_layer_norm(x, w.bfloat16())),
                      (ValueError, lambda: cw.ttt_layer_norm(x, w[:32])),
                      (ValueError, lambda: cw.ttt_layer_norm(x.t())),
                      (ValueError, lambda: cw.ttt_layer_norm(x.cpu())),
                      (TypeError, lambda: cw.ttt_layer_norm(x.half())),
                      (cw.TTTError, lambda: cw.ttt_layer_norm(x, eps=-1.0)),
                      (cw.TTTError, lambda: cw.ttt_layer_norm(x, eps=float("inf"))),
                      (cw.TTTError, lambda: cw.ttt_layer_norm(torch.zeros(1, 65544, device="cuda"))),
                      (ValueError, lambda: cw.ttt_layer_norm_backward(x, w, dy[:3], mean, rstd)),
                      (ValueError, lambda: cw.ttt_layer_norm_backward(x, w, dy, mean[:3], rstd)),
                      (ValueError, lambda: cw.ttt_layer_norm_backward(
                          x, w, dy, mean, rstd, workspace=torch.empty(4, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(err):
            call()


def test_captured_replays_equal_the_eager_calls():
    x, w, b, dy = make(513, 2560, torch.bfloat16)

    def call():
        y, mean, rstd = cw.ttt_layer_norm(x, w, b)
        return (y, mean, rstd) + cw.ttt_layer_norm_backward(x, w, dy, mean, rstd)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        x.mul_(1.25)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for s, t in zip(got, call()):
            assert torch.equal(s, t)


def test_norm_in_front_of_the_layer_and_back():
    """Hidden states x -> layer norm -> the In-Place layer; back: dO -> the layer's backward -> dH -> the norm's.  The
    gradient of x is held to the layer's own bar (fp32)."""
    cfg = ti.InplaceConfig("norm", 2, 256, 64, 136, 64, 0.05, "dot", "f32", conv_k=4, seed=3)
    t = {k: v.cuda() for k, v in ti.inplace_inputs(cfg).items()}
    x, w, b, dO = make(512, 64, torch.float32)
    x, dO = x.reshape(2, 256, 64), dO.reshape(2, 256, 64)
    H, mean, rstd = cw.ttt_layer_norm(x, w, b)
    names = ("X0", "W_gate", "W_up", "W_down0", "W_target", "conv_w")
    rest = [t[k] for k in names]
    O, _ = cw.ttt_chunk_apply_update(H, *rest, cfg.chunk, cfg.eta, "dot")
    dH = cw.ttt_layer_backward(H, *rest, dO, cfg.chunk, cfg.eta)[0]
    dx, dw, db = cw.ttt_layer_norm_backward(x, w, dH, mean, rstd)
    Hr, mr, rr = od.layer_norm(f64(x).reshape(512, 64), f64(w), f64(b))
    Hr = Hr.reshape(2, 256, 64)
    Or, _ = orc.inplace_layer(Hr, *(ti.to_f64(t[k].cpu()) for k in names), cfg.chunk, cfg.eta, "dot")
    dHr = orc.layer_backward(Hr, *(ti.to_f64(t[k].cpu()) for k in names), cfg.chunk, cfg.eta, f64(dO))[0]
    dxr, dwr, dbr = od.layer_norm_backward(f64(x).reshape(512, 64), f64(w), dHr.reshape(512, 64), mr, rr)
    assert rel(O, Or) <= 1e-4 and rel(dx.reshape(512, 64), dxr) <= 1e-4 and rel(dw, dwr) <= 1e-4 and rel(db, dbr) <= 1e-4


def test_offsets_past_32_bits():
    rows, d = 270000, 8192                          # 2.2e9 elements
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    tail, w, b, dy = make(3, d, torch.bfloat16)
    x[-3:] = tail
    y, mean, rstd = cw.ttt_layer_norm(x, w, b)
    ref = cw.ttt_layer_norm(tail, w, b)
    assert torch.equal(y[-3:], ref[0]) and torch.equal(mean[-3:], ref[1]) and torch.equal(rstd[-3:], ref[2])
    assert torch.equal(y[:2], b.expand(2, d))
    y.zero_()                                       # as dY
    y[-3:] = dy
    dx, dw, db = cw.ttt_layer_norm_backward(x, w, y, mean, rstd)
    rx, rw, rb = cw.ttt_layer_norm_backward(tail, w, dy, *ref[1:])
    assert torch.equal(dx[-3:], rx) and not dx[:2].any()
    # three rows' sums among zeros: fp32 sums of three terms in another order, 3 * 2^-24 each
    assert rel(dw, f64(rw)) <= 2.0 ** -21 and rel(db, f64(rb)) <= 2.0 ** -21
