"""Layer norm on rows of a width for every kernel variant, forward and backward, whole vectors and ragged, and the backward
pass where a workgroup has several rows.  Tolerances are those of test_gpu_norm."""
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import delta as od
from test_gpu_norm import DTYPES, SUM_TOL, TOL, f64, make, rel

pytestmark = pytest.mark.gpu

# 16-byte vectors of a row: a quarter of a wave; a wave with 1 to 8 vectors a thread; a workgroup with 1 to 16
VECTORS = [3, 16, 40, 100, 180, 250, 300, 370, 430, 500, 900, 1500, 2500, 4000, 5000, 6000, 7000, 8192, 12000, 16384]


def widths(dtype):
    V = 8 if dtype == torch.bfloat16 else 4
    return [V * n - cut for n in VECTORS for cut in (0, 3) if V * n <= 65536]


def variant(d, dtype, most):
    """(ragged, threads of a row, 0: a workgroup's, vectors a thread) of a row's kernel, as the library chooses it; a wave
    takes rows of up to 64 `most` vectors."""
    V = 8 if dtype == torch.bfloat16 else 4
    units = -(-d // V)
    tpr = 16 if units <= 16 else 64 if units <= 64 * most else 0
    nv = 1 if tpr == 16 else -(-units // (64 if tpr else 1024))
    return d % V != 0, tpr, nv if nv < 7 else 8 if nv <= 8 else 16


def every_variant(dtype, most):
    counts = {16: [1], 64: [n for n in (1, 2, 3, 4, 5, 6, 8) if n <= most],
              0: [1, 2, 3, 4, 5, 6, 8] + ([16] if dtype == torch.float32 else [])}
    return {(rag, tpr, nv) for rag in (False, True) for tpr, c in counts.items() for nv in c}


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_widths_reach_every_variant(dtype):
    for most in (8, 2):                             # forward, backward
        assert {variant(d, dtype, most) for d in widths(dtype)} == every_variant(dtype, most)


@pytest.mark.parametrize("dtype,d", [(t, d) for t in DTYPES for d in widths(t)])
def test_every_variant(dtype, d):
    rows = 21 if d < 4000 else 3
    print("norm", rows, d, dtype, variant(d, dtype, 8), variant(d, dtype, 2), flush=True)
    x, w, b, dy = make(rows, d, dtype, seed=d)
    y, mean, rstd = cw.ttt_layer_norm(x, w, b, eps=1e-4)
    yr, mr, rr = od.layer_norm(f64(x), f64(w), f64(b), 1e-4)
    assert rel(y, yr) <= TOL[dtype] and rel(mean, mr) <= 2.0 ** -17 and rel(rstd, rr) <= 2.0 ** -17
    dx, dw, db = cw.ttt_layer_norm_backward(x, w, dy, mean, rstd)
    dxr, dwr, dbr = od.layer_norm_backward(f64(x), f64(w), f64(dy), f64(mean), f64(rstd))
    assert rel(dx, dxr) <= TOL[dtype] and rel(dw, dwr) <= SUM_TOL and rel(db, dbr) <= SUM_TOL


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,d", [(30000, 64), (9000, 200), (9000, 701), (2100, 2000), (2100, 1101), (1300, 5000),
                                    (1300, 9003)])
def test_backward_with_several_rows_a_workgroup(rows, d, dtype):
    """More rows than the workgroups have places: the next row's loads are under way while one is worked on."""
    print("norm backward", rows, d, dtype, flush=True)
    x, w, _, dy = make(rows, d, dtype, seed=rows)
    mean, rstd = (torch.from_numpy(t).float().cuda() for t in od.layer_norm(f64(x))[1:])
    dx, dw, db = cw.ttt_layer_norm_backward(x, w, dy, mean, rstd)
    dxr, dwr, dbr = od.layer_norm_backward(f64(x), f64(w), f64(dy), f64(mean), f64(rstd))
    assert rel(dx, dxr) <= TOL[dtype] and rel(dw, dwr) <= SUM_TOL and rel(db, dbr) <= SUM_TOL
