"""The gated delta rule's backward at the edges of what it takes.  Tolerances are those of test_gpu_delta_backward."""
import pytest
import torch

import chunk_wise_weight_amd as cw
from test_gpu_delta import make
from test_gpu_delta_backward import B16, F32, NAMES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("n", [64, 128, 257])
def test_no_sequences(dtype, n):
    """A single start, the first entry of a longer tensor whose next one is the row's length: every gradient's rows stay
    as they are."""
    args = make(1, 1, 2, n, 64, 64, dtype, "head")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")[:1]
    outs = {x: torch.full_like(t, 7.0, dtype=dtype) for x, t in zip(NAMES, args)}
    got = cw.ttt_gated_delta_backward(*args, torch.ones_like(args[2]), seq_starts=starts, **outs)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in got[:5]) and got[5] is None
