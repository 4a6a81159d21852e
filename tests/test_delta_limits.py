"""Host-side checks of the gated delta rule's C entry points at their limits, without a GPU: what takes no workspace,
what is refused before any device work.  Pointers are never followed: any aligned address serves."""
import pytest

import chunk_wise_weight_amd as cw
from test_delta_host import shape, size

WORKSPACES = ("ttt_gated_delta_workspace_bytes", "ttt_gated_delta_backward_workspace_bytes")


@pytest.mark.parametrize("what", WORKSPACES)
@pytest.mark.parametrize("dtype", [cw.TTT_F32, cw.TTT_BF16])
def test_no_sequences_have_no_chunks(what, dtype):
    """Packed rows of no sequence: no chunk has a place, whatever the row's length (a place would be looked up behind the
    single start)."""
    for n in (0, 10, 64, 256, 1 << 20):
        assert size(shape(n=n), dtype, 0, what) == (0, 0)
    assert size(shape(n=256), dtype, 1, what)[1] > 0
