"""Host-side checks of the gated delta rule's C entry points at their limits, without a GPU: what takes no workspace,
what is refused before any device work.  Pointers are never followed: any aligned address serves."""
import ctypes

import pytest

import chunk_wise_weight_amd as cw
from test_delta_host import ARG, backward, forward, shape, size, step

WORKSPACES = ("ttt_gated_delta_workspace_bytes", "ttt_gated_delta_backward_workspace_bytes")


@pytest.mark.parametrize("what", WORKSPACES)
@pytest.mark.parametrize("dtype", [cw.TTT_F32, cw.TTT_BF16])
def test_no_sequences_have_no_chunks(what, dtype):
    """Packed rows of no sequence: no chunk has a place, whatever the row's length (a place would be looked up behind the
    single start)."""
    for n in (0, 10, 64, 256, 1 << 20):
        assert size(shape(n=n), dtype, 0, what) == (0, 0)
    assert size(shape(n=256), dtype, 1, what)[1] > 0


# Strides (batch, head, token) of a tensor [2, 2, 100, 64], and whether a written one may have them
LAYOUTS = [((12800, 6400, 64), True), ((12800, 64, 128), True), ((6400, 12800, 64), True), ((20000, 64, 160), True),
           ((64, 128, 256), True), ((12800, 6400, 0), False), ((12800, 0, 64), False), ((0, 6400, 64), False),
           ((12800, 6400, 56), False), ((12800, 32, 128), False), ((6400, 6400, 64), False), ((6400, 6336, 64), False),
           ((1 << 62, 6400, 64), False)]


@pytest.mark.parametrize("strides,apart", LAYOUTS)
def test_written_tensors_do_not_overlap_themselves(strides, apart):
    """Zero strides, and others that put two elements at one place, are for inputs only.  A call that passes the strides'
    check ends at the missing workspace, with another status than a refused one."""
    s, z, ok = shape(B=2), cw.DeltaStrides, (12800, 6400, 64)
    gate = (200, 100, 1)
    lay = cw.DeltaLayout(*(z(*ok) for _ in range(3)), z(*gate), z(*gate), z(*strides))
    opts = cw.DeltaOptions(None, None, 0, ctypes.pointer(lay))
    assert forward(s, opts=opts, ws=None) == (cw.TTT_ERR_WORKSPACE if apart else ARG)
    for at in (1, 2, 3):                                                   # dq, dk [2, 1, 100, 64], dv
        rows = [z(*ok) for _ in range(4)]
        rows[at] = z(*strides)
        fine = apart or at < 3 and strides in ((12800, 0, 64), (12800, 32, 128), (6400, 6336, 64), (6400, 6400, 64))
        got = backward(s, grads=cw.DeltaGradLayout(*rows, z(*gate), z(*gate)), ws=None)
        assert got == (cw.TTT_ERR_WORKSPACE if fine else ARG), (at, strides)
    for bad in ((200, 100, 0), (200, 0, 1), (0, 100, 1), (100, 100, 1)):
        for i in (0, 1):
            gates = [z(*gate), z(*gate)]
            gates[i] = z(*bad)
            assert backward(s, grads=cw.DeltaGradLayout(*(z(*ok) for _ in range(4)), *gates), ws=None) == ARG
    # inputs may repeat rows
    lay = cw.DeltaLayout(*(z(0, 0, 0) for _ in range(5)), z(*ok))
    assert forward(s, opts=cw.DeltaOptions(None, None, 0, ctypes.pointer(lay)), ws=None) == cw.TTT_ERR_WORKSPACE


def test_the_backward_grids_stay_below_two_to_the_32_threads():
    fwd, back = WORKSPACES
    U = cw.TTT_ERR_UNSUPPORTED
    # one workgroup of 512 a chunk and key head
    long = shape(n=(1 << 30) - 64, Hv=1, dk=8, dv=8)
    assert size(long, num=-1, what=fwd)[0] == cw.TTT_OK and size(long, num=-1, what=back)[0] == U
    assert size(shape(n=(1 << 29) - 64, Hv=1, dk=8, dv=8), what=back)[0] == cw.TTT_OK
    assert size(shape(n=(1 << 29), Hv=1, dk=8, dv=8), what=back)[0] == U
    # one of 320 each way for a sequence and value head
    many = shape(n=0, Hv=1, dk=8, dv=8)
    assert size(many, num=8000000, what=fwd)[0] == cw.TTT_OK and size(many, num=8000000, what=back)[0] == U
    assert size(many, num=6700000, what=back)[0] == cw.TTT_OK
    # shared key heads: fewer chunk workgroups for the same walks
    assert size(shape(n=(1 << 29) - 64, Hk=1, Hv=2, dk=8, dv=8), what=back)[0] == cw.TTT_OK
    assert size(shape(n=(1 << 29) - 64, Hk=2, Hv=2, dk=8, dv=8), what=back)[0] == U
    assert backward(long) == U and backward(many, opts=cw.DeltaOptions(None, 1 << 20, 8000000, None)) == U


def test_fp32_gate_gradients_are_aligned_as_such():
    lay = lambda f32: cw.DeltaGradLayout(*(cw.DeltaStrides(12800, 6400, 64) for _ in range(4)),
                                         cw.DeltaStrides(200, 100, 1), cw.DeltaStrides(200, 100, 1), f32)
    assert backward(shape(), grads=lay(0), dg=(1 << 20) + 2, ws=None) == cw.TTT_ERR_WORKSPACE
    assert backward(shape(), grads=lay(1), dg=(1 << 20) + 2, ws=None) == ARG
    assert backward(shape(), grads=lay(1), ws=None) == cw.TTT_ERR_WORKSPACE


def test_rows_that_name_their_states_are_limited():
    """Their number's square is what looking for rows of one state takes; a call past the limit is refused, one at it goes on
    to the pointers' checks."""
    U = cw.TTT_ERR_UNSUPPORTED
    assert step(R=65537, Hv=1, dv=8) == U and step(R=65536, Hv=1, dv=8, q=None) == ARG
    assert step(R=65537, S=70000, Hv=1, dv=8, slots=None, q=None) == ARG
