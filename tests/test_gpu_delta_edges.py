"""The gated delta rule, forward and step, at the edges of what it takes.  Tolerances are those of test_gpu_delta."""
import pytest
import torch

import chunk_wise_weight_amd as cw
from test_gpu_delta import DTYPES, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [64, 128, 257])
def test_no_sequences(dtype, n):
    """A single start, the first entry of a longer tensor whose next one is the row's length: no token belongs to a
    sequence, none is read, every row of O stays as it is."""
    args = make(1, 1, 2, n, 64, 64, dtype, "head")
    for t in args:
        t.fill_(float("nan"))
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")[:1]
    O = torch.full_like(args[2], 7.0)
    _, W = cw.ttt_gated_delta(*args, seq_starts=starts, O=O)
    torch.cuda.synchronize()
    assert W.shape == (0, 2, 64, 64) and (O == 7).all()
