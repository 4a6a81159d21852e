"""Idle tokens, emptied states and steep decays of the selective scan, span by span.

Each span of tokens is compared by its own norm, so that a mistake in one is not small beside the outputs of another; tokens
that empty the state have x = 0, so that what follows them has the size of what came before.  Tolerances as in
test_gpu_scan.py, which derives them; a span's outputs are sums of the same number of terms as a sequence's.
"""
import pytest
import torch

import chunk_wise_weight_amd as cw
from tests.test_gpu_scan import DTYPES, TOL_O, TOL_S, make, oracle, rel

pytestmark = pytest.mark.gpu

CUTS = [0, 17, 20, 30, 64, 70, 100, 130, 140, 170, 256, 300, 301, 350, 600]


def inputs(dtype):
    x, dt, A, B, C, D, _ = make(1, 2, 1, 600, 64, 64, dtype, "head", seed=9)
    dt = dt.abs() * 0.3
    for a, b in ((20, 30), (64, 70), (100, 130)):
        dt[:, :, a:b] = 0.0                              # idle
    dt[:, 1, 140:170] = 20.0                             # decays of e^-40 each in one head
    for h, t in ((0, 17), (0, 300), (1, 300)):
        dt[:, h, t], x[:, h, t] = 1e6, 0                 # emptied
    A[:] = torch.tensor([-1.0, -2.0])
    return (x, dt, A, B, C), D


def far(O, Or, tol):
    """The spans whose outputs are further off than they may be."""
    return [(a, b, rel(O[:, a:b], Or[:, a:b])) for a, b in zip(CUTS, CUTS[1:]) if not rel(O[:, a:b], Or[:, a:b]) <= tol]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("skip", [False, True])
def test_spans(dtype, skip):
    args, D = inputs(dtype)
    D = D if skip else None
    O, S = cw.ttt_selective_scan(*args, D=D)
    Or, Sr = oracle(0, args, D)
    assert not far(O[0], Or, TOL_O[dtype])
    assert rel(S[0], Sr) <= TOL_S
    # the state where spans end, by calls that end there; idle spans leave its bits
    states = {}
    for t in CUTS[1:]:
        cut = [v[:, :, :t] if v.dim() > 1 else v for v in args]
        states[t] = cw.ttt_selective_scan(*cut, D=D)[1]
        assert rel(states[t][0], oracle(0, args, D, cut=slice(0, t))[1]) <= TOL_S, t
    for a, b in ((20, 30), (64, 70), (100, 130)):
        assert torch.equal(states[a], states[b]), (a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_spans_find_what_is_wrong(dtype):
    """The oracle with a mistake of each kind is further off than the tolerance: rates of idle tokens, outputs left
    out."""
    args, D = inputs(dtype)
    Or, _ = oracle(0, args, D)
    for a, b in ((20, 30), (64, 70), (100, 130)):
        dt = args[1].clone()
        dt[:, :, a:b] = 0.3
        assert far(oracle(0, (args[0], dt, *args[2:]), D)[0], Or, TOL_O[dtype]), (a, b)
    for a, b in ((60, 70), (140, 170), (350, 600)):
        O = Or.copy()
        O[:, a:b] = 0
        assert far(O, Or, TOL_O[dtype]), (a, b)
