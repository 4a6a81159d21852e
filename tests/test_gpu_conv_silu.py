"""SiLU of the fp32 convolution and its derivative, value by value, far from zero too.

One tap of 1 and no bias: y = z p, p = 1 / (1 + exp(-z)), and dx = dY (p + z p (1 - p)).  exp(-|z|) is off by 2^-22 at most
(a hardware power of two good to one step, 2^-23, an argument whose rounding is put right, and two roundings), 1 + t, its
reciprocal and each product by 2^-24: 8 * 2^-24 of y.  The derivative has two terms of such factors, p (4 + 3 roundings)
and z p (1 - p) (twice that) and their sum: 16 * 2^-24 of the sum of the terms' sizes.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 61])
def test_values(d):
    z = torch.cat([torch.linspace(-80, 80, 20001), torch.randn(4000, generator=torch.Generator().manual_seed(1))])
    z = z[:len(z) // d * d].view(1, -1, d).cuda()
    w = torch.ones(d, 1, device="cuda")
    Y, _ = cw.ttt_short_conv(z, w)
    v = z.double().cpu().numpy()
    p = 1 / (1 + np.exp(-v))
    q = 1 / (1 + np.exp(v))                          # 1 - p with all its digits
    off = np.abs(Y.double().cpu().numpy() - v * p)
    print("silu", (off / np.maximum(np.abs(v * p), 1e-300)).max() * 2 ** 24, flush=True)
    assert np.all(off <= 8 * 2.0 ** -24 * np.abs(v * p))
    y1 = cw.ttt_short_conv_step(z[0], w, torch.empty(z.shape[1], 0, d, device="cuda"))
    assert torch.equal(y1, Y[0])
    dx = cw.ttt_short_conv_backward(z, w, torch.ones_like(z))[0]
    off, size = np.abs(dx.double().cpu().numpy() - (p + v * p * q)), p + np.abs(v) * p * q
    print("slope", (off / size).max() * 2 ** 24, flush=True)
    assert np.all(off <= 16 * 2.0 ** -24 * size)


def test_ends_of_the_range():
    """Where exp overflows or vanishes: y and its slope are 0 or z and 1."""
    z = torch.tensor([-3e38, -1e6, -200.0, 200.0, 1e6, 3e38, 0.0, -0.0]).view(1, 1, 8).cuda()
    w = torch.ones(8, 1, device="cuda")
    Y, _ = cw.ttt_short_conv(z, w)
    dx = cw.ttt_short_conv_backward(z, w, torch.ones_like(z))[0]
    assert torch.equal(Y[0, 0], torch.tensor([0, 0, 0, 200.0, 1e6, 3e38, 0, 0], device="cuda"))
    assert torch.equal(dx[0, 0], torch.tensor([0, 0, 0, 1, 1, 1, 0.5, 0.5], device="cuda"))
