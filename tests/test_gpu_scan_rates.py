"""Rates of the selective scan at the ends of softplus's range, on the GPU against the oracle in fp64.

softplus is 0 to fp32 below -104 and its argument above 20: a token whose dt is the type's lowest value, the usual mask, has
rate zero and leaves the state as it is, to the bit; a large rate empties it.  Tolerances as in test_gpu_scan.py and
test_gpu_scan_backward.py, which derive them.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc
from tests.test_gpu_scan import DTYPES, TOL_O, TOL_S, TOL_STEP, f64, make, rel
from tests.test_gpu_scan_backward import NAMES, tol

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min
# dt of some tokens: softplus of the first six is zero in fp32
VALUES = [LOWEST, -3e38, -2.4e38, -2.3e38, -1e38, -200.0, -104.0, -20.0, 20.0, 100.0, 1e4]
MASKS = VALUES[:6]


def masked(dtype, n, seed=0):
    """Inputs with every value of VALUES at a token of each chunk; x is zero where the rate is large, so that what follows
    has one size."""
    x, dt, A, B, C, D, bias = make(1, 4, 2, n, 64, 64, dtype, "head", seed)
    for at in range(0, n, 64):
        for i, v in enumerate(VALUES):
            t = at + 3 + 5 * i
            if t < n:
                dt[:, :, t] = v
                if v > 20:
                    x[:, :, t] = 0
    return x, dt, A, B, C, D, bias


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 60, 700])
def test_sequence_and_its_backward(dtype, n):
    print("rates", n, dtype, flush=True)
    *args, D, bias = masked(dtype, n)
    if n == 1:
        args[1][:] = LOWEST
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    S0, dS, dO = r(1, 4, 64, 64) * 0.3, r(1, 4, 64, 64), r(1, 4, n, 64).to(dtype)
    more = dict(D=D, dt_bias=bias, softplus=True, S_init=S0)
    O, S = cw.ttt_selective_scan(*args, **more)
    ref = [f64(t[0]) if t.dim() > 1 else f64(t) for t in args]
    with np.errstate(over="ignore"):
        Or, Sr = osc.selective_scan(*ref, f64(D), f64(bias), True, f64(S0[0]))
        want = osc.selective_scan_backward(*ref, f64(dO[0]), f64(D), f64(bias), True, f64(S0[0]), f64(dS[0]))
    assert rel(O[0], Or) <= TOL_O[dtype] and rel(S[0], Sr) <= TOL_S
    got = dict(zip(NAMES, cw.ttt_selective_scan_backward(*args, dO, dS_final=dS, **more)))
    at = lambda values: torch.stack([(args[1][0, 0] == v).cpu() for v in values]).any(0)
    large = at(VALUES[-3:])                          # whose dx has the rate's size: by themselves
    for k, g in got.items():
        g, w = (g[0] if g.dim() > 1 else g), want[k]
        for sel in ((large, ~large) if k == "dx" else (slice(None),)):
            if k == "dx":
                assert rel(g[:, sel], w[:, sel.numpy()]) <= tol(k, dtype), k
            else:
                assert rel(g, w) <= tol(k, dtype), k
    assert (got["ddt"][0][:, at(MASKS)] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", MASKS)
def test_masked_tokens_leave_the_state(dtype, value):
    """Nothing but masked tokens, over several segments: the state's very bits."""
    x, dt, A, B, C, D, bias = make(1, 4, 2, 900, 64, 64, dtype)
    dt[:] = value
    S0 = torch.randn(1, 4, 64, 64, generator=torch.Generator().manual_seed(1)).cuda()
    O, S = cw.ttt_selective_scan(x, dt, A, B, C, D=D, dt_bias=bias, softplus=True, S_init=S0)
    assert torch.equal(S, S0) and torch.isfinite(O).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_step(dtype):
    R = len(VALUES)
    x, dt, A, B, C, D, bias = make(1, 4, 2, R, 64, 64, dtype, seed=4)
    x, dt, B, C = (v[0].transpose(0, 1).contiguous() for v in (x, dt, B, C))
    dt[:] = torch.tensor(VALUES, device="cuda")[:, None]
    S0 = torch.randn(R, 4, 64, 64, generator=torch.Generator().manual_seed(2)).cuda()
    S = S0.clone()
    O = cw.ttt_selective_scan_step(x, dt, A, B, C, S, D=D, dt_bias=bias, softplus=True)
    for r in range(R):
        one = [f64(v[r])[:, None] if v.dim() > 1 else f64(v) for v in (x, dt, A, B, C)]
        with np.errstate(over="ignore"):
            Or, Sr = osc.selective_scan(*one, f64(D), f64(bias), True, f64(S0[r]))
        assert rel(O[r], Or[:, 0]) <= TOL_STEP[dtype] and rel(S[r], Sr) <= TOL_STEP[torch.float32], VALUES[r]
        if VALUES[r] in MASKS:
            assert torch.equal(S[r], S0[r]), VALUES[r]
