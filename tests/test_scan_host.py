"""Host-side checks of the selective scan's, short convolution's and root-mean-square norm's C entry points that need no
GPU: workspace sizes, and bad arguments refused with the documented status before any device work.  Pointers are never
followed: any aligned address serves."""
import ctypes

import pytest

import chunk_wise_weight_amd as cw
from chunk_wise_weight_amd import _lib

P = 1 << 20            # an aligned address that is not looked at
OK, ARG, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = (cw.TTT_OK, cw.TTT_ERR_ARG, cw.TTT_ERR_SHAPE, cw.TTT_ERR_DTYPE,
                                                 cw.TTT_ERR_WORKSPACE, cw.TTT_ERR_UNSUPPORTED)
Z = _lib.DeltaStrides


def shape(B=1, n=1000, H=4, G=2, P=64, N=128):
    return _lib.ScanShape(B, n, H, G, P, N)


def by(x):
    return ctypes.byref(x) if x is not None else None


def forward(s, dtype=cw.TTT_BF16, opts=None, ws=P, nbytes=1 << 40, x=P, dt=P, A=P, B=P, C=P, O=P, S=P):
    return cw.lib().ttt_selective_scan(by(s), dtype, x, dt, A, B, C, by(opts), O, S, ws, nbytes, None)


def backward(s, dtype=cw.TTT_BF16, opts=None, ws=P, nbytes=1 << 60, x=P, dt=P, A=P, B=P, C=P, O=P, S=P, grads=None, ddt=P):
    return cw.lib().ttt_selective_scan_backward(by(s), dtype, x, dt, A, B, C, O, None, by(opts), by(grads), P, ddt, S, P, P,
                                                None, None, None, ws, nbytes, None)


def size(what, s, dtype=cw.TTT_BF16, num=-1):
    out = ctypes.c_size_t(77)
    return getattr(cw.lib(), what + "_workspace_bytes")(by(s), dtype, num, ctypes.byref(out)), out.value


def options(D=None, bias=None, S0=None, starts=None, num=0, layout=None):
    return _lib.ScanOptions(D, bias, 1, S0, starts, num, ctypes.pointer(layout) if layout is not None else None)


def test_scan_workspace():
    f, b = "ttt_selective_scan", "ttt_selective_scan_backward"
    for dtype in (cw.TTT_BF16, cw.TTT_F32):
        # sequences of one segment need none, several 4 P N + 4 bytes a segment and head, in whole 16 bytes
        for s in (shape(n=0), shape(B=0), shape(n=64), shape(n=256), shape(B=300, n=512)):
            assert size(f, s, dtype) == (OK, 0)
        st, nb = size(f, shape(n=1000), dtype)
        assert st == OK and nb % (4 * (4 * 64 * 128 + 4)) == 0 and nb > 0   # whole segments of 4 heads
        assert size(b, shape(n=0), dtype) == (OK, 0)
        assert size(b, shape(n=64), dtype)[1] > 2 * 4 * 64 * 128 * 4        # two states a chunk and head
    # packed: the more sequences, the more segments
    sizes = [size(f, shape(n=4096), num=k)[1] for k in (0, 1, 5, 100)]
    assert sizes == sorted(sizes) and sizes[-1] > sizes[0]
    assert cw.lib().ttt_selective_scan_workspace_bytes(by(shape()), cw.TTT_BF16, -1, None) == ARG
    assert cw.lib().ttt_selective_scan_backward_workspace_bytes(by(shape()), cw.TTT_BF16, -1, None) == ARG


@pytest.mark.parametrize("call", [forward, backward])
def test_scan_shapes_and_arguments(call):
    for s, status in ((None, ARG), (shape(B=-1), SHAPE), (shape(n=-1), SHAPE), (shape(H=0), SHAPE), (shape(G=0), SHAPE),
                      (shape(H=3, G=2), SHAPE), (shape(P=0), SHAPE), (shape(N=0), SHAPE), (shape(P=12), UNSUPPORTED),
                      (shape(N=20), UNSUPPORTED), (shape(N=264), UNSUPPORTED), (shape(P=4104), UNSUPPORTED),
                      (shape(n=1 << 31), UNSUPPORTED), (shape(B=1 << 20, n=1 << 20), UNSUPPORTED),
                      (shape(B=1 << 31), UNSUPPORTED), (shape(n=1 << 30, H=64), UNSUPPORTED),
                      (shape(H=65544, G=1), UNSUPPORTED), (shape(B=1 << 14, n=1, H=64, P=4096, N=256), UNSUPPORTED)):
        assert call(s) == status, (s and [getattr(s, k) for k, _ in s._fields_])
    assert call(shape(), dtype=7) == DTYPE
    assert call(shape(), ws=None) == WORKSPACE and call(shape(), nbytes=10) == WORKSPACE
    assert call(shape(), ws=P + 8) == WORKSPACE
    for name in ("x", "dt", "A", "B", "C", "O", "S"):
        assert call(shape(), **{name: None}) == ARG, name
        assert call(shape(), **{name: P + 2}) == ARG, name
    for name in ("x", "B", "C", "O"):
        assert call(shape(), **{name: P + 8}) == ARG, name
    assert call(shape(B=2), opts=options(starts=P, num=3)) == SHAPE      # packed rows lie in one batch row
    assert call(shape(), opts=options(starts=P, num=-1)) == ARG
    assert call(shape(), opts=options(starts=P + 2, num=1)) == ARG
    assert call(shape(), opts=options(starts=P, num=1 << 31)) == UNSUPPORTED
    assert call(shape(), opts=options(S0=P + 4)) == ARG
    assert call(shape(), opts=options(D=P + 2)) == ARG and call(shape(), opts=options(bias=P + 1)) == ARG


def test_scan_limits():
    # (chunks + 8) heads ceil(P / 64) below 2^23, backward 2^22; states' elements by 1024 below 2^24, backward 2^23
    H = 64
    at = ((1 << 23) - 1) // H - 8
    f, b = "ttt_selective_scan", "ttt_selective_scan_backward"
    assert size(f, shape(n=64 * at, H=H))[0] == OK and size(f, shape(n=64 * (at + 1), H=H))[0] == UNSUPPORTED
    at = ((1 << 22) - 1) // H - 8
    assert size(b, shape(n=64 * at, H=H))[0] == OK and size(b, shape(n=64 * (at + 1), H=H))[0] == UNSUPPORTED
    many = shape(n=100, H=1, G=1, P=64, N=128)
    assert size(f, many, num=(1 << 21) - 8)[0] == OK and size(f, many, num=1 << 21)[0] == UNSUPPORTED
    assert size(b, many, num=(1 << 20) - 8)[0] == OK and size(b, many, num=1 << 20)[0] == UNSUPPORTED


def test_scan_strides():
    n, H, G, p, N = 1000, 4, 2, 64, 128
    good = dict(x=Z(n * H * p, p, H * p), dt=Z(n * H, 1, H), B=Z(n * G * N, N, G * N), C=Z(n * G * N, N, G * N),
                O=Z(n * H * p, p, H * p))
    # (a workspace that is too small is what a call with good strides is refused for)
    assert forward(shape(), opts=options(layout=_lib.ScanLayout(*good.values())), nbytes=1) == WORKSPACE
    for name in good:
        unit = 1 if name == "dt" else 8
        bads = [Z(0, -unit, unit), Z(0, unit, (1 << 22) + unit)] + ([Z(0, 4, 64), Z(0, 64, 60)] if unit > 1 else [])
        bads += [Z(0, 64, 0), Z(0, 0, 64), Z(0, 8, 64)] if name == "O" else []       # two elements at one place
        for bad in bads:
            lay = _lib.ScanLayout(*{**good, name: bad}.values())
            assert forward(shape(), opts=options(layout=lay)) == ARG, (name, bad.batch, bad.head, bad.token)
    # inputs may repeat
    assert forward(shape(), opts=options(layout=_lib.ScanLayout(*{**good, "x": Z(0, 0, 0)}.values())), nbytes=1) == WORKSPACE
    grads = dict(dO=good["x"], dx=good["x"], ddt=good["dt"], dB=good["B"], dC=good["B"])
    for name in grads:
        bad = Z(0, 0, 0) if name != "dO" else Z(0, -8, 8)
        assert backward(shape(), grads=_lib.ScanGradLayout(*{**grads, name: bad}.values())) == ARG, name
    assert backward(shape(), grads=_lib.ScanGradLayout(*{**grads, "dO": Z(0, 0, 0)}.values()), nbytes=1) == WORKSPACE


def scan_step(R=2, S=4, H=4, G=2, p=64, N=128, dtype=cw.TTT_BF16, x=P, dt=P, A=P, pool=P, slots=P, O=P, D=None):
    s = _lib.ScanStepShape(R, S, H, G, p, N)
    return cw.lib().ttt_selective_scan_step(by(s), dtype, x, dt, A, P, P, D, None, 1, pool, slots, O, None)


def test_scan_step():
    assert scan_step(R=0) == OK
    assert scan_step(R=-1) == SHAPE and scan_step(H=3) == SHAPE and scan_step(R=5, slots=None) == SHAPE
    assert scan_step(S=-1) == SHAPE
    assert scan_step(p=12) == UNSUPPORTED and scan_step(N=264) == UNSUPPORTED and scan_step(S=1 << 32) == UNSUPPORTED
    assert scan_step(R=65537) == UNSUPPORTED and scan_step(R=1 << 24, S=1 << 24, slots=None) == UNSUPPORTED
    assert scan_step(dtype=3) == DTYPE
    for name in ("x", "dt", "A", "pool", "O"):
        assert scan_step(**{name: None}) == ARG and scan_step(**{name: P + 2}) == ARG, name
    assert scan_step(slots=P + 2) == ARG and scan_step(D=P + 1) == ARG


def conv(B=1, n=100, d=64, K=4, dtype=cw.TTT_BF16, x=P, w=P, y=P, last=P, opts=None):
    s = _lib.ConvShape(B, n, d, K)
    return cw.lib().ttt_short_conv(by(s), dtype, x, w, by(opts), y, last, None)


def conv_options(bias=None, x0=None, starts=None, num=0, layout=None):
    return _lib.ConvOptions(bias, 1, x0, starts, num, ctypes.pointer(layout) if layout is not None else None)


def conv_backward(B=1, n=100, d=64, K=4, dtype=cw.TTT_BF16, dy=P, dx=P, dw=P, opts=None, grads=None, ws=P, nbytes=1 << 40):
    s = _lib.ConvShape(B, n, d, K)
    return cw.lib().ttt_short_conv_backward(by(s), dtype, P, P, dy, None, by(opts), by(grads), dx, dw, None, None, ws,
                                            nbytes, None)


def test_conv():
    R = _lib.RowStrides
    for call in (conv, conv_backward):
        assert call(B=-1) == SHAPE and call(n=-1) == SHAPE and call(d=0) == SHAPE and call(K=0) == SHAPE
        assert call(K=9) == UNSUPPORTED and call(d=(1 << 20) + 1) == UNSUPPORTED and call(n=1 << 31) == UNSUPPORTED
        assert call(B=1 << 16, n=1 << 16) == UNSUPPORTED and call(dtype=5) == DTYPE
        assert call(B=2, opts=conv_options(starts=P, num=3)) == SHAPE
        assert call(opts=conv_options(starts=P, num=-1)) == ARG and call(opts=conv_options(starts=P + 2, num=1)) == ARG
        assert call(opts=conv_options(starts=P, num=1 << 31)) == UNSUPPORTED
        assert call(opts=conv_options(bias=P + 1)) == ARG and call(opts=conv_options(x0=P + 1)) == ARG
        for bad in (R(-1, 64), R(0, -64), R(0, (1 << 40) + 1)):
            assert call(opts=conv_options(layout=_lib.ConvLayout(bad, R(6400, 64)))) == ARG
    for bad in (R(6400, 63), R(6400, 0)):
        assert conv(opts=conv_options(layout=_lib.ConvLayout(R(0, 0), bad))) == ARG
    assert conv(B=2, opts=conv_options(layout=_lib.ConvLayout(R(0, 0), R(0, 64)))) == ARG
    for name in ("x", "w", "y", "last"):
        assert conv(**{name: None}) == ARG and conv(**{name: P + 1}) == ARG, name
    for name in ("dy", "dx", "dw"):
        assert conv_backward(**{name: None}) == ARG and conv_backward(**{name: P + 1}) == ARG, name
    assert conv_backward(grads=_lib.ConvGradLayout(R(0, 0), R(6400, 0))) == ARG
    assert conv_backward(ws=None) == WORKSPACE and conv_backward(nbytes=8) == WORKSPACE and conv_backward(ws=P + 4) == WORKSPACE
    s = _lib.ConvShape(1, 100, 64, 4)
    st, nb = size("ttt_short_conv_backward", s)
    assert st == OK and nb > 0 and nb % (5 * 64 * 4) == 0
    assert size("ttt_short_conv_backward", _lib.ConvShape(1, 0, 64, 4)) == (OK, 0)
    assert cw.lib().ttt_short_conv_backward_workspace_bytes(by(s), cw.TTT_BF16, -1, None) == ARG


def conv_step(R=2, S=4, d=64, K=4, dtype=cw.TTT_BF16, x=P, w=P, halo=P, slots=P, y=P):
    return cw.lib().ttt_short_conv_step(R, S, d, K, dtype, 1, x, w, None, halo, slots, y, None)


def test_conv_step():
    assert conv_step(R=0) == OK
    assert conv_step(R=-1) == SHAPE and conv_step(d=0) == SHAPE and conv_step(R=5, slots=None) == SHAPE
    assert conv_step(K=9) == UNSUPPORTED and conv_step(R=65537) == UNSUPPORTED and conv_step(S=1 << 32) == UNSUPPORTED
    assert conv_step(dtype=3) == DTYPE and conv_step(slots=P + 2) == ARG
    for name in ("x", "w", "halo", "y"):
        assert conv_step(**{name: None}) == ARG and conv_step(**{name: P + 1}) == ARG, name


def rms(rows=4, dim=64, dtype=cw.TTT_BF16, eps=1e-5, x=P, res=None, w=P, h=P, y=P, rstd=P, scale=None, group=0):
    return cw.lib().ttt_rms_norm(rows, dim, dtype, eps, x, res, w, h, y, rstd, scale, group, None)


def test_rms_norm():
    assert rms(rows=0) == OK
    assert rms(rows=-1) == SHAPE and rms(dim=0) == SHAPE and rms(dim=65537) == UNSUPPORTED
    assert rms(dtype=9) == DTYPE and rms(eps=-1.0) == ARG and rms(eps=float("nan")) == ARG
    for name in ("x", "y", "rstd"):
        assert rms(**{name: None}) == ARG and rms(**{name: P + 2}) == ARG, name
    assert rms(w=P + 8) == ARG and rms(res=P + 2) == ARG and rms(res=P, h=None) == ARG
    assert rms(group=128) == ARG and rms(scale=P, group=48) == ARG and rms(scale=P, group=-1) == ARG
    assert rms(scale=P + 2) == ARG
    out = ctypes.c_size_t(0)
    f = cw.lib().ttt_rms_norm_backward_workspace_bytes
    assert f(0, 64, cw.TTT_F32, ctypes.byref(out)) == OK and out.value == 0
    assert f(7, 1001, cw.TTT_F32, ctypes.byref(out)) == OK and out.value % (1001 * 4) == 0 and out.value > 0
    assert f(7, 1001, cw.TTT_F32, None) == ARG
    g = cw.lib().ttt_rms_norm_backward
    assert g(4, 64, cw.TTT_BF16, P, P, P, P, P, P, P, None, 0, None) == WORKSPACE
    assert g(4, 64, cw.TTT_BF16, P, P, None, P, P, P, P, P, 1 << 30, None) == ARG
    assert g(4, 64, cw.TTT_BF16, P, P, P, P, P + 8, P, P, P, 1 << 30, None) == ARG
