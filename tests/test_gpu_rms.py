"""Root-mean-square norm of a sum, in 8 bits too, and its backward on the GPU against the oracle in fp64.

Tolerances (relative Frobenius norm, unless said otherwise).  A rounding is off by half a step: bf16 2^-8, fp32 2^-24,
e4m3 2^-4 of the value (2^-10 below 2^-6).
  sums    fp32 sums of up to 2^16 terms, kept by each thread over at most 64 and joined in a tree, 2^7 roundings of
          2^-24 deep: 2^-17 at most.
  H       one rounding of the sum.  bf16 sums are rounded to fp32 first: where that meets a tie the second rounding
          may go the other way, still at most half a step and 2^-24 off.
  Y       the sums' error and one rounding to Y's type.
  scale   the sums' error and a few roundings of fp32.
  e4m3    values lie on a grid; y / scale is off by 2^-16 of itself, so each value is one of the grid's two nearest to
          the exact one and at most (2^-4 + 2^-15) of it (2^-10 below 2^-6) off.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SUMS = 2.0 ** -17
DTYPES = [torch.float32, torch.bfloat16]
E4M3 = torch.float8_e4m3fn


def rel(a, b):
    n = np.linalg.norm(b)
    a = a.double().cpu().numpy()
    return float(np.linalg.norm(a - b) / n) if n else float(np.abs(a).max(initial=0.0))


def f64(x):
    return None if x is None else x.double().cpu().numpy()


# rows and widths of every variant: parts of a wave, waves, workgroups; whole vectors and not
SIZES = [(1, 8), (5, 128), (1, 1), (37, 100), (3, 512), (9, 1001), (4, 1536), (6, 2560), (300, 264), (2, 4096), (3, 5000),
         (2, 8192), (2, 9001), (1, 16384), (2, 20000), (1, 65536), (1, 40001), (2000, 72)]


def make(rows, d, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    x = (r(rows, d) * (0.5 + torch.rand(rows, 1, generator=gen))).to(dtype).cuda()
    return (x, (3 * r(rows, d)).to(dtype).cuda(), (1 + 0.3 * r(d)).to(dtype).cuda(), r(rows, d).to(dtype).cuda(),
            r(rows, d).to(dtype).cuda())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", SIZES)
def test_forward_and_backward(size, dtype):
    rows, d = size
    print("rms", size, dtype, flush=True)
    x, res, w, dy, dh = make(rows, d, dtype)
    for weight, residual, back in ((w, res, dh), (w, None, None), (None, res, None), (None, None, dh)):
        Y, H, rstd, scale = cw.ttt_rms_norm(x, weight, residual, eps=1e-4)
        assert scale is None and Y.dtype == dtype
        if residual is None:
            assert H is x
        else:
            assert rel(H, f64(x) + f64(res)) <= HALF[dtype] + 2.0 ** -24
        yr, rr = osc.rms_norm(f64(H), f64(weight), 1e-4)
        assert rel(Y, yr) <= HALF[dtype] + SUMS and rel(rstd, rr) <= SUMS
        dx, dw = cw.ttt_rms_norm_backward(H, weight, dy, rstd, dH=back)
        dxr, dwr = osc.rms_norm_backward(f64(H), f64(weight), f64(dy), f64(rstd), f64(back))
        if d > 2 or back is not None:    # a row of one: dx is zero but for roundings
            assert rel(dx, dxr) <= HALF[dtype] + SUMS
        assert (dw is None) == (weight is None)
        assert dw is None or rel(dw, dwr) <= SUMS


def check_e4m3(Y, scale, H, weight, eps, group):
    """Every value and scale of an 8-bit output against the oracle."""
    yr, _ = osc.rms_norm(f64(H), f64(weight), eps)
    sr = osc.scales(yr, group)
    s = f64(scale).reshape(sr.shape)
    assert np.all(np.abs(s - sr) <= 2.0 ** -16 * sr)
    q = yr / np.repeat(sr, group or yr.shape[1], 1)[:, :yr.shape[1]]
    got = Y.float().double().cpu().numpy()
    assert np.all(np.isfinite(got)) and np.array_equal(osc.e4m3(got), got)
    assert np.all(np.abs(got - q) <= np.maximum((2.0 ** -4 + 2.0 ** -15) * np.abs(q), 2.0 ** -10 + 2.0 ** -20))
    # rounding is monotone: the result lies between those of the values 2^-15 to either side, which differ from the
    # nearest only next to a tie (of bf16 rows without a weight, q is 448 times a ratio of 8-bit numbers: ties are common)
    low, high = osc.e4m3(q * (1 - 2.0 ** -15)), osc.e4m3(np.clip(q * (1 + 2.0 ** -15), -448, 448))
    assert np.all((got == low) | (got == high))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [None, 32, 64, 128])
@pytest.mark.parametrize("size", SIZES)
def test_8_bits(size, group, dtype):
    rows, d = size
    print("rms e4m3", size, group, dtype, flush=True)
    x, res, w, _, _ = make(rows, d, dtype, 1)
    for weight, residual in ((w, res), (None, None)):
        Y, H, rstd, scale = cw.ttt_rms_norm(x, weight, residual, eps=1e-4, out_dtype=E4M3, group=group)
        assert Y.dtype == E4M3 and tuple(scale.shape) == ((rows,) if group is None else (rows, -(-d // group)))
        check_e4m3(Y, scale, H, weight, 1e-4, group)


@pytest.mark.parametrize("dtype", DTYPES)
def test_8_bits_of_zero_tiny_and_far_apart_values(dtype):
    """Rows of zeros have the least scale and zero values; a group's scale follows its own columns."""
    x = torch.zeros(4, 256, dtype=dtype, device="cuda")
    x[1, :128] = 1e-3
    x[1, 200] = 1000.0
    x[2, 5] = 2.0 ** -60
    x[3] = torch.arange(256) - 128.0
    for group in (None, 32, 128):
        Y, H, rstd, scale = cw.ttt_rms_norm(x, eps=1e-6, out_dtype=E4M3, group=group)
        assert (Y[0].float() == 0).all() and (scale[0] == 2.0 ** -126).all()
        check_e4m3(Y, scale, H, None, 1e-6, group)
        assert Y[3].float().abs().max() == 448


@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_against_differences(dtype):
    """The gradient of sum(Y dY) along a direction against central differences of the oracle at the same H: dx and the
    difference's own error of some eps^2 third derivatives; fp64 differences at 1e-4 are exact to 1e-6."""
    x, _, w, dy, dh = make(3, 100, dtype, 7)
    Y, H, rstd, _ = cw.ttt_rms_norm(x, w)
    dx, dw = cw.ttt_rms_norm_backward(H, w, dy, rstd, dH=dh)
    step = np.random.default_rng(1).normal(size=(3, 100))
    loss = lambda h: (osc.rms_norm(h, f64(w))[0] * f64(dy)).sum() + (h * f64(dh)).sum()
    diff = (loss(f64(H) + 1e-4 * step) - loss(f64(H) - 1e-4 * step)) / 2e-4
    tol = (HALF[dtype] + SUMS) * np.linalg.norm(f64(dx)) * np.linalg.norm(step) + 1e-6
    assert abs((f64(dx) * step).sum() - diff) <= tol


def test_unaligned_rows_no_rows_and_given_outputs():
    x, res, w, dy, _ = make(6, 333, torch.bfloat16)
    flat = torch.zeros(6 * 333 + 1, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:].view(6, 333).copy_(x)                     # rows of 333 need their elements' alignment only
    a, b = cw.ttt_rms_norm(x, w, res), cw.ttt_rms_norm(odd, w, res)
    assert all(torch.equal(s, t) for s, t in zip(a[:3], b[:3]))
    # batches of any leading sizes, outputs in place
    Y, H = torch.empty(2, 3, 333, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 3, 333, dtype=torch.bfloat16, device="cuda")
    c = cw.ttt_rms_norm(x.view(2, 3, 333), w, res.view(2, 3, 333), Y=Y, H=H)
    assert c[0] is Y and c[1] is H and torch.equal(Y.view(6, 333), a[0]) and c[2].shape == (2, 3)
    empty = x[:0]
    Y, H, rstd, scale = cw.ttt_rms_norm(empty, w, empty, out_dtype=E4M3, group=32)
    assert Y.shape == (0, 333) and scale.shape == (0, 11)
    dx, dw = cw.ttt_rms_norm_backward(empty, w, empty, rstd)
    assert dx.shape == (0, 333) and (dw == 0).all()


def test_other_rows_do_not_reach_a_row():
    """Rows of NaN and infinities leave the others' bits alone."""
    x, res, w, _, _ = make(40, 264, torch.float32)
    good = cw.ttt_rms_norm(x, w, res, out_dtype=E4M3)
    x2 = x.clone()
    x2[::3] = float("nan")
    x2[1::3, 5] = float("inf")
    bad = cw.ttt_rms_norm(x2, w, res, out_dtype=E4M3)
    for s, t in zip(good, bad):
        assert torch.equal(s[2::3].contiguous().view(torch.uint8), t[2::3].contiguous().view(torch.uint8))


def test_refusals():
    x, res, w, dy, _ = make(4, 64, torch.bfloat16)
    for bad in (dict(residual=res[:, :32]), dict(residual=res.float()), dict(weight=w.float()), dict(weight=w[:32]),
                dict(out_dtype=torch.float16), dict(group=32), dict(out_dtype=E4M3, group=16), dict(scale=w.float()),
                dict(Y=dy.t()), dict(residual=res.cpu())):
        with pytest.raises((ValueError, TypeError)):
            cw.ttt_rms_norm(x, **bad)
    with pytest.raises(cw.TTTError):
        cw.ttt_rms_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        cw.ttt_rms_norm_backward(x, w, dy, torch.zeros(3, device="cuda"))
