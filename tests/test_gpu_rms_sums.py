"""The root-mean-square norm's weight gradient: a sum over all rows that keeps small terms next to large ones.

h and rstd are 1, so that a row's term is dY itself, and dY holds whole numbers: 2^24 in some rows, -2^24 in others, 1
between them (next to 2^24 a 1 is lost in fp32).  The sum is exact in fp64 and a small whole number: nothing may differ.
"""
import pytest
import torch

import chunk_wise_weight_amd as cw

pytestmark = pytest.mark.gpu

BIG = 2.0 ** 24
DTYPES = [torch.float32, torch.bfloat16]


def gradient(dY):
    rows, d = dY.shape
    ones = torch.ones(rows, d, dtype=dY.dtype, device="cuda")
    dw = cw.ttt_rms_norm_backward(ones, torch.ones(d, dtype=dY.dtype, device="cuda"), dY, torch.ones(rows, device="cuda"))[1]
    return dw


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [1, 40, 72, 512, 1001, 2560, 5000, 16384])
def test_rows_far_apart(d, dtype):
    """One term in 16 rows: every workgroup's own sum is exact, theirs has to be."""
    print("rms sums", d, dtype, flush=True)
    dY = torch.zeros(704, d, dtype=dtype, device="cuda")
    dY[::16] = 1
    dY[0], dY[688] = BIG, -BIG
    assert (gradient(dY) == 42).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,d", [(768 * 3, 2560), (1280 * 4 * 3, 320), (1280 * 16 * 3, 40), (768 * 5, 5000)])
def test_rows_of_a_thread(rows, d, dtype):
    """A third of the rows has 2^24, the next 1, the last -2^24: a workgroup takes rows of all three."""
    print("rms sums", rows, d, dtype, flush=True)
    third = rows // 3
    dY = torch.empty(rows, d, dtype=dtype, device="cuda")
    dY[:third], dY[third:2 * third], dY[2 * third:] = BIG, 1, -BIG
    assert (gradient(dY) == third).all()
