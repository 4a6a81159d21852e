"""Decays inside a chunk of the bf16 selective scan behind tokens that empty the state.

Each emptying token adds -173 (base 2) to the chunk's running sum of log decays, 48 of them -8310: differences of such sums
in one fp32 are off by up to 2^-10, their powers by 2^-10.5, which rounds outputs to the wrong bf16 value once in twenty or
so.  With decays good to 2^-16 and products to 2^-16 the value before its rounding is off by 2^-15 at most, and a result
differs from the rounded exact one where a border between two values (2^-8 apart at least) lies that near: for 2 * 2^-15 /
2^-8 = 2^-6 of them.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc
from tests.test_gpu_scan import f64, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64), (32, 200), (64, 16)])
@pytest.mark.parametrize("shared", [1, 2])
def test_outputs_are_the_rounded_ones(P, N, shared):
    H, n = 2 * shared, 64 * 9
    print("decays", H, P, N, flush=True)
    x, dt, A, B, C, _, _ = make(1, H, 2, n, P, N, torch.bfloat16, "head", seed=3)
    # one token feeds the state, those behind it read it: outputs of one term, whose error is the decay's
    A[:] = -1.0
    dt[:] = 200.0
    x[:] = 0
    read = torch.zeros(n, dtype=torch.bool)
    for c in range(0, n, 64):
        x[:, :, c + 48] = torch.randn(H, P, generator=torch.Generator().manual_seed(c)).to(x.dtype).cuda()
        dt[:, :, c + 48:c + 64] = 0.01 + 0.3 * torch.rand(H, 16, generator=torch.Generator().manual_seed(c + 1)).cuda()
        read[c + 48:c + 64] = True
    O, _ = cw.ttt_selective_scan(x, dt, A, B, C)
    Or, _ = osc.selective_scan(*(f64(t[0]) if t.dim() > 1 else f64(t) for t in (x, dt, A, B, C)))
    want = torch.from_numpy(Or).to(torch.bfloat16)[:, read]
    got = O[0].cpu()[:, read]
    # C . B of a token near zero cancels: only outputs whose terms do not are counted
    cb = np.einsum("gcn,gcin->gci", f64(B[0])[:, 48::64], f64(C[0]).reshape(2, n // 64, 64, N)[:, :, 48:])
    size = np.einsum("gcn,gcin->gci", np.abs(f64(B[0]))[:, 48::64], np.abs(f64(C[0]).reshape(2, n // 64, 64, N)[:, :, 48:]))
    sound = torch.from_numpy(np.abs(cb) > size / 8).flatten(1).repeat_interleave(shared, 0)
    assert sound.float().mean() > 0.1
    wrong = (got != want)[sound].float().mean().item()
    print("wrong", wrong, "bound", 2.0 ** -6, flush=True)
    assert wrong <= 2.0 ** -6
