"""Host-side checks of the gated delta rule's and layer norm's C entry points that need no GPU: workspace sizes, and bad
arguments refused with the documented status before any device work.  Pointers are never followed: any aligned address
serves."""
import ctypes

import pytest

import chunk_wise_weight_amd as cw

P = 1 << 20            # an aligned address that is not looked at
ARG, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = (cw.TTT_ERR_ARG, cw.TTT_ERR_SHAPE, cw.TTT_ERR_DTYPE, cw.TTT_ERR_WORKSPACE,
                                             cw.TTT_ERR_UNSUPPORTED)


def shape(B=1, n=100, Hk=1, Hv=2, dk=64, dv=64):
    return cw.DeltaShape(B, n, Hk, Hv, dk, dv)


def forward(s, dtype=cw.TTT_BF16, scale=1.0, opts=None, q=P, ws=P, nbytes=1 << 40, W=P):
    opts = ctypes.byref(opts) if opts is not None else None
    return cw.lib().ttt_gated_delta(ctypes.byref(s), dtype, scale, q, P, P, P, P, opts, P, W, ws, nbytes, None)


def backward(s, dtype=cw.TTT_BF16, scale=1.0, opts=None, dO=P, ws=P, nbytes=1 << 40, grads=None, dg=P):
    opts = ctypes.byref(opts) if opts is not None else None
    grads = ctypes.byref(grads) if grads is not None else None
    return cw.lib().ttt_gated_delta_backward(ctypes.byref(s), dtype, scale, P, P, P, P, P, dO, None, opts, grads, P, P, P,
                                             dg, P, None, ws, nbytes, None)


def size(s, dtype=cw.TTT_BF16, num=-1, what="ttt_gated_delta_workspace_bytes"):
    out = ctypes.c_size_t(0)
    return getattr(cw.lib(), what)(ctypes.byref(s), dtype, num, ctypes.byref(out)), out.value


def test_workspace_sizes():
    # a chunk and head: 6 fragments each of T (hi, lo) and P, 1 KB of gates; fp32: 10 of T, 10 of P
    assert size(shape(n=100)) == (0, 2 * 2 * (18 * 1024 + 1024))
    assert size(shape(n=100), cw.TTT_F32) == (0, 2 * 2 * (20 * 1024 + 1024))
    assert size(shape(n=0)) == (0, 0) and size(shape(B=0)) == (0, 0)
    # packed: n / 64 + sequences chunk slots
    assert size(shape(n=100), num=5) == (0, (1 + 5) * 2 * 19 * 1024)
    st, nb = size(shape(n=64), what="ttt_gated_delta_backward_workspace_bytes")
    assert st == 0 and nb == 2 * (19 * 1024 + 25 * 1024 + 2 * 64 * 64 * 2 + 2 * 64 * 64 * 2)


@pytest.mark.parametrize("call", [forward, backward])
def test_shapes_and_arguments(call):
    for s, status in ((shape(B=-1), SHAPE), (shape(n=-1), SHAPE), (shape(Hk=0), SHAPE), (shape(Hk=2, Hv=3), SHAPE),
                      (shape(dk=12), UNSUPPORTED), (shape(dk=264), UNSUPPORTED), (shape(dv=20), UNSUPPORTED),
                      (shape(dv=4104), UNSUPPORTED), (shape(n=1 << 31), UNSUPPORTED), (shape(B=1 << 20, n=1 << 20), UNSUPPORTED),
                      (shape(n=1 << 30, Hv=64, Hk=64), UNSUPPORTED)):
        assert call(s) == status
    assert call(shape(), dtype=7) == DTYPE
    assert call(shape(), scale=float("nan")) == ARG and call(shape(), scale=float("inf")) == ARG
    assert call(shape(), ws=None) == WORKSPACE and call(shape(), nbytes=10) == WORKSPACE
    assert call(shape(), ws=P + 8) == WORKSPACE
    opts = cw.DeltaOptions(None, P, 3, None)
    assert call(shape(B=2), opts=opts) == SHAPE                          # packed rows lie in one batch row
    assert call(shape(), opts=cw.DeltaOptions(None, P, -1, None)) == ARG
    assert call(shape(), opts=cw.DeltaOptions(None, P + 2, 1, None)) == ARG
    assert call(shape(), opts=cw.DeltaOptions(P + 4, None, 0, None)) == ARG


def test_strides():
    z = cw.DeltaStrides
    for bad in (z(0, -64, 64), z(0, 64, 65), z(0, 60, 64), z(0, 64, (1 << 22) + 64)):
        lay = cw.DeltaLayout(bad, *(z(0, 6400, 64) for _ in range(5)))
        assert forward(shape(), opts=cw.DeltaOptions(None, None, 0, ctypes.pointer(lay))) == ARG
    lay = cw.DeltaGradLayout(*(z(0, 6400, 64) for _ in range(3)), z(0, 6400, -64), z(), z())
    assert backward(shape(), grads=lay) == ARG


def test_pointers():
    assert forward(shape(), q=None) == ARG and forward(shape(), q=P + 8) == ARG and forward(shape(), W=None) == ARG
    assert backward(shape(), dO=None) == ARG and backward(shape(), dg=P + 1) == ARG


def step(R=2, S=4, Hk=1, Hv=2, dk=64, dv=64, dtype=cw.TTT_BF16, scale=1.0, slots=P, W=P, q=P):
    s = cw.DeltaStepShape(R, S, Hk, Hv, dk, dv)
    return cw.lib().ttt_gated_delta_step(ctypes.byref(s), dtype, scale, q, P, P, P, P, W, slots, P, None)


def test_step():
    assert step(R=0) == cw.TTT_OK
    assert step(R=-1) == SHAPE and step(Hv=3, Hk=2) == SHAPE and step(R=5, slots=None) == SHAPE
    assert step(dk=260) == UNSUPPORTED and step(R=1 << 24) == UNSUPPORTED and step(S=1 << 32) == UNSUPPORTED
    assert step(dtype=3) == DTYPE and step(scale=float("inf")) == ARG
    assert step(W=None) == ARG and step(q=None) == ARG and step(slots=P + 2) == ARG


def norm(rows=4, dim=64, dtype=cw.TTT_BF16, eps=1e-5, x=P, w=P, mean=P):
    return cw.lib().ttt_layer_norm(rows, dim, dtype, eps, x, w, P, P, mean, P, None)


def test_norm():
    assert norm(rows=0) == cw.TTT_OK
    assert norm(rows=-1) == SHAPE and norm(dim=0) == SHAPE and norm(dim=65537) == UNSUPPORTED
    assert norm(dtype=9) == DTYPE and norm(eps=-1.0) == ARG and norm(eps=float("nan")) == ARG
    assert norm(x=None) == ARG and norm(x=P + 2) == ARG and norm(w=P + 8) == ARG and norm(mean=None) == ARG
    out = ctypes.c_size_t(0)
    f = cw.lib().ttt_layer_norm_backward_workspace_bytes
    assert f(0, 64, cw.TTT_F32, ctypes.byref(out)) == 0 and out.value == 0
    assert f(7, 1001, cw.TTT_F32, ctypes.byref(out)) == 0 and out.value % (2 * 1001 * 4) == 0 and out.value > 0
    assert f(7, 1001, cw.TTT_F32, None) == ARG
    g = cw.lib().ttt_layer_norm_backward
    assert g(4, 64, cw.TTT_BF16, P, P, P, P, P, P, P, P, None, 0, None) == WORKSPACE
    assert g(4, 64, cw.TTT_BF16, P, P, None, P, P, P, P, P, P, 1 << 30, None) == ARG
