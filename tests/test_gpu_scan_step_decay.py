"""The decay of the selective scan's token step, value by value: exp(A r) far from zero keeps its digits.

x is zero and A r exact, so that the state is S exp(A r): a power of two good to one step (2^-23), its argument's rounding
put right to first order, two roundings there and one of the product: 6 * 2^-24.  A product below 2^-126, as exp(-85) =
1.2e-37 times an element below 0.1, is a multiple of 2^-149 whatever its size and off by half of that: 2^-150 more."""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decays(dtype):
    R, H, P, N = 680, 2, 8, 8
    rate = (torch.arange(R) / 8.0 + 0.125)[:, None].expand(R, H).contiguous().cuda()       # 1/8 .. 85
    A = torch.tensor([-1.0, -0.5], device="cuda")
    S0 = torch.randn(R, H, P, N, generator=torch.Generator().manual_seed(1)).cuda()
    S = S0.clone()
    z = lambda *s: torch.zeros(*s, dtype=dtype, device="cuda")
    cw.ttt_selective_scan_step(z(R, H, P), rate, A, z(R, 1, N), z(R, 1, N), S)
    a = np.exp(A.double().cpu().numpy() * rate.double().cpu().numpy())[:, :, None, None]
    want = S0.double().cpu().numpy() * a
    off = np.abs(S.double().cpu().numpy() - want) - 2.0 ** -150
    print("decay", (off / np.abs(want)).max() * 2 ** 24, flush=True)
    assert np.all(off <= 6 * 2.0 ** -24 * np.abs(want))
