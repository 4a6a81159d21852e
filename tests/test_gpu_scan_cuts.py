"""Packed rows whose sequences are cut into segments, some of them, on workspaces that hold NaN: what a call has not written
it does not read.  Against the oracle, with the tolerances of test_gpu_scan.py and test_gpu_scan_backward.py."""
import pytest
import torch

import chunk_wise_weight_amd as cw
from tests.test_gpu_scan import DTYPES, TOL_O, TOL_S, make, oracle, rel
from tests.test_gpu_scan_backward import check, reference

pytestmark = pytest.mark.gpu

LENS = [[1500, 0, 64, 2000, 1, 1, 700, 300], [5000], [1] * 40 + [3000] + [1] * 40, [0, 129, 0, 2001, 0]]


def nan(nbytes):
    return torch.full((nbytes // 4 + 1,), float("nan"), device="cuda")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", LENS)
def test_packed(dtype, lens):
    H, G, P, N, front, behind = 4, 2, 32, 16, 37, 70
    n, num = front + sum(lens) + behind, len(lens)
    print("cuts", lens, dtype, flush=True)
    *args, D, bias = make(1, H, G, n, P, N, dtype, seed=num)
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    dO, S0, dS = r(1, n, H, P).to(dtype).transpose(1, 2), r(num, H, P, N) * 0.3, r(num, H, P, N)
    starts = torch.tensor([front] + lens).cumsum(0).to(torch.int32).cuda()
    shape = cw._lib.ScanShape(1, n, H, G, P, N)
    fwd = cw.ttt_selective_scan_workspace_bytes(shape, dtype, num)
    bwd = cw.ttt_selective_scan_backward_workspace_bytes(shape, dtype, num)
    assert fwd > 0
    more = dict(D=D, dt_bias=bias, softplus=True, S_init=S0, seq_starts=starts)
    O, S = cw.ttt_selective_scan(*args, workspace=nan(fwd), **more)
    parts, at = [], front
    for m in lens:
        parts.append((0, slice(at, at + m)))
        at += m
    for i, (_, cut) in enumerate(parts):
        Or, Sr = oracle(0, args, D, bias, True, S0[i], cut)
        assert rel(O[0, :, cut], Or) <= TOL_O[dtype] and rel(S[i], Sr) <= TOL_S, i
    grads = cw.ttt_selective_scan_backward(*args, dO, dS_final=dS, workspace=nan(bwd), **more)
    ref, total = reference(args, dO, D, bias, True, S0, dS, parts)
    check(grads, ref, total, parts, dtype, S0, D, bias)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_batch_of_cut_rows(dtype):
    B, H, G, n, P, N = 3, 2, 1, 1700, 64, 32
    *args, D, bias = make(B, H, G, n, P, N, dtype)
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    dO, S0, dS = r(B, n, H, P).to(dtype).transpose(1, 2), r(B, H, P, N) * 0.3, r(B, H, P, N)
    shape = cw._lib.ScanShape(B, n, H, G, P, N)
    fwd = cw.ttt_selective_scan_workspace_bytes(shape, dtype)
    bwd = cw.ttt_selective_scan_backward_workspace_bytes(shape, dtype)
    assert fwd > 0
    more = dict(D=D, dt_bias=bias, softplus=True, S_init=S0)
    O, S = cw.ttt_selective_scan(*args, workspace=nan(fwd), **more)
    for b in range(B):
        Or, Sr = oracle(b, args, D, bias, True, S0[b])
        assert rel(O[b], Or) <= TOL_O[dtype] and rel(S[b], Sr) <= TOL_S, b
    grads = cw.ttt_selective_scan_backward(*args, dO, dS_final=dS, workspace=nan(bwd), **more)
    parts = [(b, slice(None)) for b in range(B)]
    ref, total = reference(args, dO, D, bias, True, S0, dS, parts)
    check(grads, ref, total, parts, dtype, S0, D, bias)
