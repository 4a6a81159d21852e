"""How many digits the selective scan keeps, where that can be told: results of one token, and of positive terms alone.

One token from a zero state.  S = (r x) B^T: r x is rounded once in fp32 and enters products with all its 24 bits, so a
state's element is off by that rounding and its own, 2 * 2^-24, and twice that for the sum of the parts: a part of the value
left out would be 2^-17 of it.
Positive terms do not cancel, so that every relative error stays below the number of roundings that a term passes, here at
most N + P of sums over features, 64 of a chunk's tokens twice, 5 chunks of states and 32 of factors.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc
from tests.test_gpu_scan import DTYPES, f64, make, rel
from tests.test_gpu_scan_backward import NAMES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,G,P,N", [(4, 2, 64, 128), (2, 2, 40, 200), (6, 1, 16, 16)])
def test_state_of_one_token(H, G, P, N, dtype):
    print("one token", H, G, P, N, dtype, flush=True)
    x, dt, A, B, C, _, _ = make(3, H, G, 1, P, N, dtype, seed=2)
    dt = dt.abs()
    _, S = cw.ttt_selective_scan(x, dt, A, B, C)
    Bh = f64(B[:, :, 0]).repeat(H // G, 1)
    want = (f64(dt[:, :, 0])[..., None] * f64(x[:, :, 0]))[..., None] * Bh[:, :, None]
    off = np.abs(f64(S) - want) / np.maximum(np.abs(want), 1e-300)
    print("state", off.max() * 2 ** 24, flush=True)
    assert off.max() <= 4 * 2.0 ** -24


@pytest.mark.parametrize("dtype", DTYPES)
def test_positive_terms(dtype):
    H, G, P, N, n = 4, 2, 16, 16, 300
    x, dt, A, B, C, D, _ = make(1, H, G, n, P, N, dtype, "head", seed=5)
    x, B, C, D, dt = x.abs(), B.abs(), C.abs(), D.abs(), dt.abs() * 0.2
    dO = torch.randn(x.shape, generator=torch.Generator().manual_seed(6)).abs().to(dtype).cuda()
    args = (x, dt, A, B, C)
    ref = [f64(t[0]) if t.dim() > 1 else f64(t) for t in args]
    O, S = cw.ttt_selective_scan(*args, D=D)
    Or, Sr = osc.selective_scan(*ref, f64(D))
    want = osc.selective_scan_backward(*ref, f64(dO[0]), f64(D))
    got = dict(zip(NAMES, cw.ttt_selective_scan_backward(*args, dO, D=D)))
    got, want = {**{k: v for k, v in got.items() if v is not None}, "O": O, "S": S}, {**want, "O": Or, "S": Sr}
    fp32 = (N + P + 2 * 64 + 5 + 32) * 2.0 ** -24
    pairs = 2.0 ** -8 + 4 * 2.0 ** -16               # bf16 outputs: their rounding, and products of pairs of bf16 values
    for k, g in got.items():
        if k in ("ddt", "ddt_bias"):                 # A is negative: these do cancel
            continue
        g = g[0] if g.dim() > 1 else g
        tol = fp32 if g.dtype == torch.float32 else pairs
        print(k, rel(g, want[k]) * 2 ** 24, tol * 2 ** 24, flush=True)
        assert rel(g, want[k]) <= tol, k
