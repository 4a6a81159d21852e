"""The short convolution's sums over tokens (dconv_w, dbias) keep small terms next to large ones.

x and its earlier rows are 1 and there is no SiLU, so that a token's term is dY itself for the bias and every tap; dY holds
whole numbers at tokens 1024 apart: 2^24 at the first, -2^24 at the last, 1 between them (next to 2^24 a 1 is lost in fp32).
No run of a thread (at most 64 tokens) and no workgroup's runs next to one another hold two of them where channels are 64
vectors and more; the sum is exact in fp64 and a small whole number: nothing may differ.
"""
import pytest
import torch

import chunk_wise_weight_amd as cw

pytestmark = pytest.mark.gpu

BIG = 2.0 ** 24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("d,K", [(256, 4), (1024, 4), (257, 3), (512, 8), (300, 1)])
def test_tokens_far_apart(d, K, packed, dtype):
    n, step = 128 * 1024, 1024
    print("conv sums", d, K, packed, dtype, flush=True)
    x = torch.ones(1, n, d, dtype=dtype, device="cuda")
    dY = torch.zeros_like(x)
    dY[:, ::step] = 1
    dY[:, 0], dY[:, n - step] = BIG, -BIG
    starts = torch.tensor([0, 5000, 5000, n], dtype=torch.int32, device="cuda") if packed else None
    x0 = torch.ones(3 if packed else 1, K - 1, d, dtype=dtype, device="cuda")
    _, dw, db, _ = cw.ttt_short_conv_backward(x, x.new_ones(d, K), dY, x.new_ones(d), silu=False, x_init=x0, seq_starts=starts)
    assert (dw == n // step - 2).all() and (db == n // step - 2).all()
