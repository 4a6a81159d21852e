"""The 8-bit output of the root-mean-square norm, code by code: y / scale as its definition has it, each operation rounded to
fp32 and the quotient rounded once more, to e4m3.  Every operation is exact to half a step, so nothing may differ."""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [None, 32, 64, 128])
@pytest.mark.parametrize("small", [0, -100, -110, -120])
@pytest.mark.parametrize("rows,d", [(300, 2560), (41, 1001), (700, 40), (5, 20000)])
def test_codes_are_the_rounded_quotients(rows, d, group, dtype, small):
    """small: exponents of the weight, down to scales at their least, 2^-126."""
    print("rms e4m3", rows, d, group, dtype, small, flush=True)
    gen = torch.Generator().manual_seed(rows + d)
    x = torch.randn(rows, d, generator=gen).to(dtype).cuda()
    w = ((1 + 0.3 * torch.randn(d, generator=gen)) * 2.0 ** small).to(dtype).cuda()
    Y, H, rstd, scale = cw.ttt_rms_norm(x, w, eps=1e-4, out_dtype=E4M3, group=group)
    f32 = lambda t: t.float().cpu().numpy()
    y = f32(x) * f32(rstd)[:, None] * f32(w)
    assert y.dtype == np.float32
    g = group or d
    parts = [y[:, i:i + g] for i in range(0, d, g)]
    s = np.stack([np.maximum(np.abs(p).max(-1) / np.float32(448), np.float32(2.0 ** -126)) for p in parts], -1)
    assert np.array_equal(f32(scale).reshape(s.shape), s)
    q = np.concatenate([p / s[:, i:i + 1] for i, p in enumerate(parts)], -1)
    assert q.dtype == np.float32
    assert np.array_equal(f32(Y), osc.e4m3(q.astype(np.float64)))
