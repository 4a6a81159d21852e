"""ctypes marshalling for libttt.so.  No arithmetic of the layer happens here:
the functions check that the tensors they are given match the shape they
declare (the C ABI sees only raw pointers), allocate outputs and workspace
with torch on the tensors' device, and pass pointers and the current stream."""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libttt.so")

(TTT_OK, TTT_ERR_ARG, TTT_ERR_SHAPE, TTT_ERR_DTYPE, TTT_ERR_WORKSPACE, TTT_ERR_DEVICE, TTT_ERR_UNSUPPORTED,
 TTT_ERR_SCRATCH_LIMIT) = range(8)
TTT_NOALLOC_SCRATCH_BYTES = 64 << 20     # the static scratch of ttt_chunk_apply_update_noalloc
TTT_F32, TTT_BF16 = 0, 1
TTT_MODE_DOT, TTT_MODE_MSE, TTT_MODE_DOT_SCAN = 0, 1, 2
TTT_UPDATE_THEN_APPLY, TTT_APPLY_THEN_UPDATE = 0, 1

_MODES = {"dot": TTT_MODE_DOT, "mse": TTT_MODE_MSE, "dot_scan": TTT_MODE_DOT_SCAN}
_ORDERS = {"update_then_apply": TTT_UPDATE_THEN_APPLY, "apply_then_update": TTT_APPLY_THEN_UPDATE}
_DTYPES = {torch.float32: TTT_F32, torch.bfloat16: TTT_BF16}


class InplaceShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seq_len", "d_model", "d_ff", "chunk", "conv_k")]


class LayerOptions(ctypes.Structure):
    _fields_ = [("doc_starts", ctypes.c_void_p), ("conv_forward", ctypes.c_int), ("W_init", ctypes.c_void_p),
                ("x0_halo", ctypes.c_void_p), ("W_states", ctypes.c_void_p), ("update_mask", ctypes.c_void_p),
                ("update_first", ctypes.c_int)]


class LactOptions(ctypes.Structure):
    _fields_ = [("order", ctypes.c_int), ("update_mask", ctypes.c_void_p), ("eta_tok", ctypes.c_void_p),
                ("loss", ctypes.c_int), ("weight_norm", ctypes.c_int), ("muon", ctypes.c_int),
                ("side_stream", ctypes.c_void_p), ("fork_event", ctypes.c_void_p), ("join_event", ctypes.c_void_p),
                ("W_states", ctypes.c_void_p)]


class LactSideStream:
    """A side stream and the fork / join events that let ttt_lact_swiglu run its (batch, head) rows as two chains
    (the caller owns all three; the library creates none).  Create it outside graph capture and keep it alive while
    calls that use it may run; calls that may be enqueued concurrently need one each."""

    def __init__(self, device=None):
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.device = dev
        self.stream = torch.cuda.Stream(device=dev)
        self.fork = torch.cuda.Event()
        self.join = torch.cuda.Event()
        # torch creates an event's handle at its first record
        self.fork.record(self.stream)
        self.join.record(self.stream)
        self.stream.synchronize()

    def handles(self):
        return (ctypes.c_void_p(self.stream.cuda_stream), ctypes.c_void_p(self.fork.cuda_event),
                ctypes.c_void_p(self.join.cuda_event))


class BackwardOptions(ctypes.Structure):
    _fields_ = [("W_states", ctypes.c_void_p), ("doc_starts", ctypes.c_void_p), ("update_mask", ctypes.c_void_p),
                ("conv_forward", ctypes.c_int), ("W_init", ctypes.c_void_p), ("x0_halo", ctypes.c_void_p),
                ("dW_init", ctypes.c_void_p), ("dx0_halo", ctypes.c_void_p)]


class LactShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "heads", "seq_len", "head_dim", "hidden", "chunk")]


class DeltaShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seq_len", "k_heads", "v_heads", "k_dim", "v_dim")]


class DeltaStepShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "states", "k_heads", "v_heads", "k_dim", "v_dim")]


class DeltaStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "head", "token")]


class DeltaLayout(ctypes.Structure):
    _fields_ = [(n, DeltaStrides) for n in ("q", "k", "v", "g", "beta", "O")]


class DeltaGradLayout(ctypes.Structure):
    _fields_ = [(n, DeltaStrides) for n in ("dO", "dq", "dk", "dv", "dg", "dbeta")] + [("gates_f32", ctypes.c_int)]


class DeltaOptions(ctypes.Structure):
    _fields_ = [("W_init", ctypes.c_void_p), ("seq_starts", ctypes.c_void_p), ("num_seqs", ctypes.c_int64),
                ("layout", ctypes.POINTER(DeltaLayout))]


class ConvShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seq_len", "dim", "taps")]


class RowStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "token")]


class ConvLayout(ctypes.Structure):
    _fields_ = [(n, RowStrides) for n in ("x", "y")]


class ConvGradLayout(ctypes.Structure):
    _fields_ = [(n, RowStrides) for n in ("dy", "dx")]


class ConvOptions(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("silu", ctypes.c_int), ("x_init", ctypes.c_void_p),
                ("seq_starts", ctypes.c_void_p), ("num_seqs", ctypes.c_int64), ("layout", ctypes.POINTER(ConvLayout))]


class ScanShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seq_len", "heads", "groups", "head_dim", "state")]


class ScanLayout(ctypes.Structure):
    _fields_ = [(n, DeltaStrides) for n in ("x", "dt", "B", "C", "O")]


class ScanGradLayout(ctypes.Structure):
    _fields_ = [(n, DeltaStrides) for n in ("dO", "dx", "ddt", "dB", "dC")]


class ScanOptions(ctypes.Structure):
    _fields_ = [("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("softplus", ctypes.c_int),
                ("S_init", ctypes.c_void_p), ("seq_starts", ctypes.c_void_p), ("num_seqs", ctypes.c_int64),
                ("layout", ctypes.POINTER(ScanLayout))]


class ScanStepShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "states", "heads", "groups", "head_dim", "state")]


class TTTError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)}")
        self.status = status


_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_S = ctypes.c_size_t
_SIGNATURES = {
    "ttt_status_string": (ctypes.c_char_p, [_I]),
    "ttt_inplace_workspace_bytes": (_I, [ctypes.POINTER(InplaceShape), _I, _I, _I, ctypes.POINTER(_S)]),
    "ttt_chunk_apply_update": (_I, [ctypes.POINTER(InplaceShape), _I, _I, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _S, _P]),
    "ttt_chunk_apply_update_ex": (_I, [ctypes.POINTER(InplaceShape), _I, _I, _F, _P, _P, _P, _P, _P, _P, _P,
                                       ctypes.POINTER(LayerOptions), _P, _P, _P, _S, _P]),
    "ttt_chunk_apply_update_noalloc": (_I, [ctypes.POINTER(InplaceShape), _I, _I, _F] + [_P] * 10),
    "ttt_core_apply_update": (_I, [ctypes.POINTER(InplaceShape), _I, _I, _F, _P, _P, _P, _P, _P, _P, _S, _P]),
    "ttt_core_apply_update_ex": (_I, [ctypes.POINTER(InplaceShape), _I, _I, _F, _P, _P, _P,
                                      ctypes.POINTER(LayerOptions), _P, _P, _P, _S, _P]),
    "ttt_core_backward_workspace_bytes": (_I, [ctypes.POINTER(InplaceShape), _I, _I, ctypes.POINTER(_S)]),
    "ttt_core_backward_mse_workspace_bytes": (_I, [ctypes.POINTER(InplaceShape), _I, _I, ctypes.POINTER(_S)]),
    "ttt_core_backward_mse": (_I, [ctypes.POINTER(InplaceShape), _I, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                   _S, _P]),
    "ttt_layer_backward_workspace_bytes": (_I, [ctypes.POINTER(InplaceShape), _I, _I, ctypes.POINTER(_S)]),
    "ttt_layer_backward": (_I, [ctypes.POINTER(InplaceShape), _I, _F] + [_P] * 18 + [_S, _P]),
    "ttt_layer_backward_mse_workspace_bytes": (_I, [ctypes.POINTER(InplaceShape), _I, _I, ctypes.POINTER(_S)]),
    "ttt_layer_backward_ex": (_I, [ctypes.POINTER(InplaceShape), _I, _I, _F] + [_P] * 8 +
                              [ctypes.POINTER(BackwardOptions)] + [_P] * 7 + [_P, _S, _P]),
    "ttt_core_backward_ex": (_I, [ctypes.POINTER(InplaceShape), _I, _I, _F, _P, _P, _P, _P,
                                  ctypes.POINTER(BackwardOptions), _P, _P, _P, _P, _S, _P]),
    "ttt_layer_backward_mse": (_I, [ctypes.POINTER(InplaceShape), _I, _F] + [_P] * 18 + [_S, _P]),
    "ttt_core_backward": (_I, [ctypes.POINTER(InplaceShape), _I, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S,
                               _P]),
    "ttt_produce_z": (_I, [ctypes.POINTER(InplaceShape), _I, _P, _P, _P, _P, _P, _P]),
    "ttt_vhat_workspace_bytes": (_I, [ctypes.POINTER(InplaceShape), _I, ctypes.POINTER(_S)]),
    "ttt_produce_vhat": (_I, [ctypes.POINTER(InplaceShape), _I, _F, _P, _P, _P, _P, _P, _S, _P]),
    "ttt_chunk_delta": (_I, [ctypes.POINTER(InplaceShape), _I, _P, _P, _P, _P]),
    "ttt_chunk_scan": (_I, [ctypes.POINTER(InplaceShape), _I, _F, _P, _P, _P, _P, _P]),
    "ttt_update_scan_workspace_bytes": (_I, [ctypes.POINTER(InplaceShape), _I, ctypes.POINTER(_S)]),
    "ttt_chunk_update_scan": (_I, [ctypes.POINTER(InplaceShape), _I, _P, _P, _P, _P, _P, _P, _S, _P]),
    "ttt_chunk_apply": (_I, [ctypes.POINTER(InplaceShape), _I, _P, _P, _P, _P]),
    "ttt_lact_workspace_bytes": (_I, [ctypes.POINTER(LactShape), _I, ctypes.POINTER(_S)]),
    "ttt_lact_swiglu": (_I, [ctypes.POINTER(LactShape), _I, _I, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                             _S, _P]),
    "ttt_lact_swiglu_ex": (_I, [ctypes.POINTER(LactShape), _I, _F, _P, _P, _P, _P, _P, _P,
                                ctypes.POINTER(LactOptions), _P, _P, _P, _P, _P, _S, _P]),
    "ttt_lact_backward_workspace_bytes": (_I, [ctypes.POINTER(LactShape), _I, ctypes.POINTER(_S)]),
    "ttt_lact_backward_workspace_bytes_ex": (_I, [ctypes.POINTER(LactShape), _I, _I, ctypes.POINTER(_S)]),
    "ttt_lact_swiglu_backward": (_I, [ctypes.POINTER(LactShape), _I, _I, _F] + [_P] * 13 + [_P, _S, _P]),
    "ttt_lact_swiglu_backward_ex": (_I, [ctypes.POINTER(LactShape), _I, _F] + [_P] * 7 +
                                    [ctypes.POINTER(LactOptions)] + [_P] * 6 + [_P, _S, _P]),
    "ttt_gated_delta_workspace_bytes": (_I, [ctypes.POINTER(DeltaShape), _I, ctypes.c_int64, ctypes.POINTER(_S)]),
    "ttt_gated_delta": (_I, [ctypes.POINTER(DeltaShape), _I, _F] + [_P] * 5 + [ctypes.POINTER(DeltaOptions)] +
                        [_P] * 3 + [_S, _P]),
    "ttt_gated_delta_backward_workspace_bytes": (_I, [ctypes.POINTER(DeltaShape), _I, ctypes.c_int64,
                                                      ctypes.POINTER(_S)]),
    "ttt_gated_delta_backward": (_I, [ctypes.POINTER(DeltaShape), _I, _F] + [_P] * 7 +
                                 [ctypes.POINTER(DeltaOptions), ctypes.POINTER(DeltaGradLayout)] + [_P] * 7 + [_S, _P]),
    "ttt_gated_delta_step": (_I, [ctypes.POINTER(DeltaStepShape), _I, _F] + [_P] * 9),
    "ttt_layer_norm": (_I, [ctypes.c_int64, ctypes.c_int64, _I, _F] + [_P] * 7),
    "ttt_layer_norm_backward_workspace_bytes": (_I, [ctypes.c_int64, ctypes.c_int64, _I, ctypes.POINTER(_S)]),
    "ttt_layer_norm_backward": (_I, [ctypes.c_int64, ctypes.c_int64, _I] + [_P] * 9 + [_S, _P]),
    "ttt_rms_norm": (_I, [ctypes.c_int64, ctypes.c_int64, _I, _F] + [_P] * 7 + [ctypes.c_int64, _P]),
    "ttt_rms_norm_backward_workspace_bytes": (_I, [ctypes.c_int64, ctypes.c_int64, _I, ctypes.POINTER(_S)]),
    "ttt_rms_norm_backward": (_I, [ctypes.c_int64, ctypes.c_int64, _I] + [_P] * 8 + [_S, _P]),
    "ttt_short_conv": (_I, [ctypes.POINTER(ConvShape), _I, _P, _P, ctypes.POINTER(ConvOptions), _P, _P, _P]),
    "ttt_short_conv_backward_workspace_bytes": (_I, [ctypes.POINTER(ConvShape), _I, ctypes.c_int64, ctypes.POINTER(_S)]),
    "ttt_short_conv_backward": (_I, [ctypes.POINTER(ConvShape), _I] + [_P] * 4 + [ctypes.POINTER(ConvOptions),
                                     ctypes.POINTER(ConvGradLayout)] + [_P] * 5 + [_S, _P]),
    "ttt_short_conv_step": (_I, [ctypes.c_int64] * 4 + [_I, _I] + [_P] * 7),
    "ttt_selective_scan_workspace_bytes": (_I, [ctypes.POINTER(ScanShape), _I, ctypes.c_int64, ctypes.POINTER(_S)]),
    "ttt_selective_scan": (_I, [ctypes.POINTER(ScanShape), _I] + [_P] * 5 + [ctypes.POINTER(ScanOptions)] + [_P] * 3 +
                           [_S, _P]),
    "ttt_selective_scan_backward_workspace_bytes": (_I, [ctypes.POINTER(ScanShape), _I, ctypes.c_int64,
                                                         ctypes.POINTER(_S)]),
    "ttt_selective_scan_backward": (_I, [ctypes.POINTER(ScanShape), _I] + [_P] * 7 + [ctypes.POINTER(ScanOptions),
                                         ctypes.POINTER(ScanGradLayout)] + [_P] * 9 + [_S, _P]),
    "ttt_selective_scan_step": (_I, [ctypes.POINTER(ScanStepShape), _I] + [_P] * 7 + [_I] + [_P] * 4),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libttt.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"{lib_path} is missing: build it with `python -m chunk_wise_weight_amd.build`")
        handle = ctypes.CDLL(lib_path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def exported_symbols():
    return list(_SIGNATURES)


def status_string(status: int) -> str:
    return lib().ttt_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != TTT_OK:
        raise TTTError(status, what)


def _dt(dtype: torch.dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    return _DTYPES[dtype]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _vp(t):
    """A tensor's address, or None for a missing or empty tensor."""
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() else None


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: torch.Tensor, name: str, shape, dtype, device):
    if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_cuda and t.device == device
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (the layer runs only in the HIP library)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _mode(mode) -> int:
    if isinstance(mode, str):
        return _MODES[mode]
    return int(mode)


def _inplace_shape(B, n, d, f, chunk, K) -> InplaceShape:
    return InplaceShape(int(B), int(n), int(d), int(f), int(chunk), int(K))


def _flags(t, name, shape, dev):
    """A per-chunk flag tensor (bool or uint8, device) as uint8, or None."""
    if t is None:
        return None
    if t.dtype == torch.bool:
        t = t.to(torch.uint8)
    _need(t, name, shape, torch.uint8, dev)
    return t


def ttt_inplace_workspace_bytes(shape: InplaceShape, dtype: torch.dtype, mode="dot", with_producers=True) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_inplace_workspace_bytes(ctypes.byref(shape), _dt(dtype), _mode(mode), int(bool(with_producers)),
                                             ctypes.byref(out)), "ttt_inplace_workspace_bytes")
    return out.value


def _workspace(nbytes: int, device, workspace):
    if workspace is not None:
        if workspace.device.type != "cuda" or workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def ttt_chunk_apply_update(H, X0, W_gate, W_up, W_down0, W_target, conv_w, chunk: int, eta: float, mode="dot",
                           O=None, W_final=None, workspace=None, doc_starts=None, conv_forward=False, W_init=None,
                           x0_halo=None, W_states=None, update_mask=None, update_first=False):
    """The whole In-Place layer.  Returns (O [B, n, d], W_final [B, d, f] fp32).

    Options (ttt_chunk_apply_update_ex): doc_starts, a uint8 (or bool) device tensor [B, seq_len // chunk] whose
    nonzero entries mark the chunks that start a new document in their row; conv_forward, the forward-looking
    in-chunk convolution for the target; W_init [B, d, f] fp32 and x0_halo [B, K-1, d] to resume rows from an
    earlier call (its W_final and its last K-1 rows of X0); W_states [B, seq_len // chunk, d, f] (dtype) to keep
    the per-chunk states of the dot objective for ttt_core_backward; update_mask, a uint8 (or bool) device tensor
    [B, seq_len // chunk] whose zero entries mark chunks that are applied without updating the state;
    update_first, each chunk's step taken before its apply (every mode; not with W_states)."""
    B, n, d = H.shape
    f = W_gate.shape[0]
    K = conv_w.shape[1]
    dt, dev = H.dtype, H.device
    for name, t, shp in (("H", H, (B, n, d)), ("X0", X0, (B, n, d)), ("W_gate", W_gate, (f, d)),
                         ("W_up", W_up, (f, d)), ("W_down0", W_down0, (d, f)), ("W_target", W_target, (d, d)),
                         ("conv_w", conv_w, (d, K))):
        _need(t, name, shp, dt, dev)
    shape = _inplace_shape(B, n, d, f, chunk, K)
    O = torch.empty(B, n, d, dtype=dt, device=dev) if O is None else O
    W_final = torch.empty(B, d, f, dtype=torch.float32, device=dev) if W_final is None else W_final
    _need(O, "O", (B, n, d), dt, dev)
    _need(W_final, "W_final", (B, d, f), torch.float32, dev)
    nbytes = ttt_inplace_workspace_bytes(shape, dt, mode, True)
    ws = _workspace(nbytes, dev, workspace)
    if W_init is not None:
        _need(W_init, "W_init", (B, d, f), torch.float32, dev)
    if x0_halo is not None:
        _need(x0_halo, "x0_halo", (B, K - 1, d), dt, dev)
    if W_states is not None:
        _need(W_states, "W_states", (B, n // chunk, d, f), dt, dev)
    update_mask = _flags(update_mask, "update_mask", (B, n // chunk if chunk > 0 else 0), dev)
    if doc_starts is None and not conv_forward and W_init is None and x0_halo is None and W_states is None and \
            update_mask is None and not update_first:
        _check(lib().ttt_chunk_apply_update(ctypes.byref(shape), _dt(dt), _mode(mode), float(eta), _ptr(H),
                                            _ptr(X0), _ptr(W_gate), _ptr(W_up), _ptr(W_down0), _ptr(W_target),
                                            _ptr(conv_w), _ptr(O), _ptr(W_final), _ptr(ws), nbytes, _stream(dev)),
               "ttt_chunk_apply_update")
        return O, W_final
    if doc_starts is not None:
        if doc_starts.dtype == torch.bool:
            doc_starts = doc_starts.to(torch.uint8)
        _need(doc_starts, "doc_starts", (B, n // chunk if chunk > 0 else 0), torch.uint8, dev)
    ptr = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() > 0 else None
    opts = LayerOptions(ptr(doc_starts), 1 if conv_forward else 0, ptr(W_init), ptr(x0_halo), ptr(W_states),
                        ptr(update_mask), 1 if update_first else 0)
    _check(lib().ttt_chunk_apply_update_ex(ctypes.byref(shape), _dt(dt), _mode(mode), float(eta), _ptr(H),
                                           _ptr(X0), _ptr(W_gate), _ptr(W_up), _ptr(W_down0), _ptr(W_target),
                                           _ptr(conv_w), ctypes.byref(opts), _ptr(O), _ptr(W_final), _ptr(ws),
                                           nbytes, _stream(dev)),
           "ttt_chunk_apply_update_ex")
    return O, W_final


def ttt_chunk_apply_update_noalloc(H, X0, W_gate, W_up, W_down0, W_target, conv_w, chunk: int, eta: float, mode,
                                   O, W_final):
    """The whole In-Place layer into the caller's O [B, n, d] and W_final [B, d, f] (fp32), with its scratch taken
    from the library's static device buffer (TTT_NOALLOC_SCRATCH_BYTES): nothing is allocated here or in the
    library.  Raises TTTError with TTT_ERR_SCRATCH_LIMIT for shapes whose scratch does not fit.  Returns (O,
    W_final)."""
    B, n, d = H.shape
    f = W_gate.shape[0]
    K = conv_w.shape[1]
    dt, dev = H.dtype, H.device
    for name, t, shp in (("H", H, (B, n, d)), ("X0", X0, (B, n, d)), ("W_gate", W_gate, (f, d)),
                         ("W_up", W_up, (f, d)), ("W_down0", W_down0, (d, f)), ("W_target", W_target, (d, d)),
                         ("conv_w", conv_w, (d, K)), ("O", O, (B, n, d))):
        _need(t, name, shp, dt, dev)
    _need(W_final, "W_final", (B, d, f), torch.float32, dev)
    shape = _inplace_shape(B, n, d, f, chunk, K)
    _check(lib().ttt_chunk_apply_update_noalloc(ctypes.byref(shape), _dt(dt), _mode(mode), float(eta), _ptr(H),
                                                _ptr(X0), _ptr(W_gate), _ptr(W_up), _ptr(W_down0), _ptr(W_target),
                                                _ptr(conv_w), _ptr(O), _ptr(W_final), _stream(dev)),
           "ttt_chunk_apply_update_noalloc")
    return O, W_final


def ttt_core_apply_update(Z, Vhat, W_down0, chunk: int, eta: float, mode="dot", O=None, W_final=None,
                          workspace=None, W_states=None, update_mask=None, doc_starts=None, W_init=None,
                          update_first=False):
    """The chunk loop given Z [B, n, f] and Vhat [B, n, d].  Returns (O, W_final).  W_states [B, n // chunk, d, f]
    (dtype), if given, receives the per-chunk states; update_mask and doc_starts [B, n // chunk], W_init
    [B, d, f] fp32 and update_first as for the layer (all through ttt_core_apply_update_ex)."""
    B, n, f = Z.shape
    d = Vhat.shape[2]
    dt, dev = Z.dtype, Z.device
    _need(Z, "Z", (B, n, f), dt, dev)
    _need(Vhat, "Vhat", (B, n, d), dt, dev)
    _need(W_down0, "W_down0", (d, f), dt, dev)
    shape = _inplace_shape(B, n, d, f, chunk, 1)
    O = torch.empty(B, n, d, dtype=dt, device=dev) if O is None else O
    W_final = torch.empty(B, d, f, dtype=torch.float32, device=dev) if W_final is None else W_final
    _need(O, "O", (B, n, d), dt, dev)
    _need(W_final, "W_final", (B, d, f), torch.float32, dev)
    nbytes = ttt_inplace_workspace_bytes(shape, dt, mode, False)
    ws = _workspace(nbytes, dev, workspace)
    update_mask = _flags(update_mask, "update_mask", (B, n // chunk if chunk > 0 else 0), dev)
    doc_starts = _flags(doc_starts, "doc_starts", (B, n // chunk if chunk > 0 else 0), dev)
    if W_states is not None or update_mask is not None or doc_starts is not None or W_init is not None or \
            update_first:
        if W_states is not None:
            _need(W_states, "W_states", (B, n // chunk, d, f), dt, dev)
        if W_init is not None:
            _need(W_init, "W_init", (B, d, f), torch.float32, dev)
        opts = LayerOptions(_vp(doc_starts), 0, _vp(W_init), None, _vp(W_states), _vp(update_mask),
                            1 if update_first else 0)
        _check(lib().ttt_core_apply_update_ex(ctypes.byref(shape), _dt(dt), _mode(mode), float(eta), _ptr(Z),
                                              _ptr(Vhat), _ptr(W_down0), ctypes.byref(opts), _ptr(O), _ptr(W_final),
                                              _ptr(ws), nbytes, _stream(dev)),
               "ttt_core_apply_update_ex")
        return O, W_final
    _check(lib().ttt_core_apply_update(ctypes.byref(shape), _dt(dt), _mode(mode), float(eta), _ptr(Z), _ptr(Vhat),
                                       _ptr(W_down0), _ptr(O), _ptr(W_final), _ptr(ws), nbytes, _stream(dev)),
           "ttt_core_apply_update")
    return O, W_final


def ttt_core_backward_workspace_bytes(shape: InplaceShape, dtype: torch.dtype, saved_states=False) -> int:
    n = ctypes.c_size_t()
    _check(lib().ttt_core_backward_workspace_bytes(ctypes.byref(shape), _dt(dtype), int(bool(saved_states)),
                                                   ctypes.byref(n)),
           "ttt_core_backward_workspace_bytes")
    return n.value


def _core_backward(mode, Z, Vhat, W_down0, dO, chunk, eta, dZ, dVhat, dW_down0, workspace, W_states, doc_starts,
                   update_mask, W_init):
    B, n, f = Z.shape
    d = Vhat.shape[2]
    dt, dev = Z.dtype, Z.device
    _need(Z, "Z", (B, n, f), dt, dev)
    _need(Vhat, "Vhat", (B, n, d), dt, dev)
    _need(W_down0, "W_down0", (d, f), dt, dev)
    _need(dO, "dO", (B, n, d), dt, dev)
    shape = _inplace_shape(B, n, d, f, chunk, 1)
    dZ = torch.empty(B, n, f, dtype=dt, device=dev) if dZ is None else dZ
    dVhat = torch.empty(B, n, d, dtype=dt, device=dev) if dVhat is None else dVhat
    dW_down0 = torch.empty(d, f, dtype=torch.float32, device=dev) if dW_down0 is None else dW_down0
    _need(dZ, "dZ", (B, n, f), dt, dev)
    _need(dVhat, "dVhat", (B, n, d), dt, dev)
    _need(dW_down0, "dW_down0", (d, f), torch.float32, dev)
    k = n // chunk if chunk > 0 else 0
    if W_states is not None:
        _need(W_states, "W_states", (B, k, d, f), dt, dev)
    dW_init = None
    if W_init is not None:
        _need(W_init, "W_init", (B, d, f), torch.float32, dev)
        dW_init = torch.empty(B, d, f, dtype=torch.float32, device=dev)
    nbytes = (ttt_core_backward_mse_workspace_bytes if mode == "mse" else ttt_core_backward_workspace_bytes)(
        shape, dt, W_states is not None)
    ws = _workspace(nbytes, dev, workspace)
    sp = _vp(W_states)
    doc_starts = _flags(doc_starts, "doc_starts", (B, k), dev)
    dp = _vp(doc_starts)
    if update_mask is not None or W_init is not None:
        um = _flags(update_mask, "update_mask", (B, k), dev)
        opts = BackwardOptions(sp, dp, _vp(um), 0, _vp(W_init), None, _vp(dW_init), None)
        _check(lib().ttt_core_backward_ex(ctypes.byref(shape), _dt(dt), _mode(mode), float(eta), _ptr(Z), _ptr(Vhat),
                                          _ptr(W_down0), _ptr(dO), ctypes.byref(opts), _ptr(dZ), _ptr(dVhat),
                                          _ptr(dW_down0), _ptr(ws), nbytes, _stream(dev)), "ttt_core_backward_ex")
    else:
        name = "ttt_core_backward_mse" if mode == "mse" else "ttt_core_backward"
        _check(getattr(lib(), name)(ctypes.byref(shape), _dt(dt), float(eta), _ptr(Z), _ptr(Vhat), _ptr(W_down0),
                                    _ptr(dO), sp, dp, _ptr(dZ), _ptr(dVhat), _ptr(dW_down0), _ptr(ws), nbytes,
                                    _stream(dev)), name)
    return (dZ, dVhat, dW_down0) if W_init is None else (dZ, dVhat, dW_down0, dW_init)


def ttt_core_backward(Z, Vhat, W_down0, dO, chunk: int, eta: float, dZ=None, dVhat=None, dW_down0=None,
                      workspace=None, W_states=None, doc_starts=None, update_mask=None, W_init=None):
    """Gradients through the dot chunk loop given dO = dLoss/dO [B, n, d], with the per-chunk states W_states
    [B, n // chunk, d, f] kept by the forward call, or recomputed (None); doc_starts [B, n // chunk] packs documents,
    update_mask [B, n // chunk] masks updates and W_init [B, d, f] fp32 resumes rows as for the forward layer (the
    last two through ttt_core_backward_ex).  Returns (dZ [B, n, f], dVhat [B, n, d], dW_down0 [d, f] fp32), and
    dW_init [B, d, f] fp32 after them when W_init is given."""
    return _core_backward("dot", Z, Vhat, W_down0, dO, chunk, eta, dZ, dVhat, dW_down0, workspace, W_states,
                          doc_starts, update_mask, W_init)


def ttt_core_backward_mse_workspace_bytes(shape: InplaceShape, dtype: torch.dtype, saved_states=False) -> int:
    n = ctypes.c_size_t()
    _check(lib().ttt_core_backward_mse_workspace_bytes(ctypes.byref(shape), _dt(dtype), int(bool(saved_states)),
                                                       ctypes.byref(n)),
           "ttt_core_backward_mse_workspace_bytes")
    return n.value


def ttt_core_backward_mse(Z, Vhat, W_down0, dO, chunk: int, eta: float, dZ=None, dVhat=None, dW_down0=None,
                          workspace=None, W_states=None, doc_starts=None, update_mask=None, W_init=None):
    """ttt_core_backward for the MSE chunk loop (same arguments and results)."""
    return _core_backward("mse", Z, Vhat, W_down0, dO, chunk, eta, dZ, dVhat, dW_down0, workspace, W_states,
                          doc_starts, update_mask, W_init)


def ttt_layer_backward_workspace_bytes(shape: InplaceShape, dtype: torch.dtype, saved_states=False,
                                       mode="dot") -> int:
    n = ctypes.c_size_t()
    name = "ttt_layer_backward_mse_workspace_bytes" if mode == "mse" else "ttt_layer_backward_workspace_bytes"
    _check(getattr(lib(), name)(ctypes.byref(shape), _dt(dtype), int(bool(saved_states)), ctypes.byref(n)), name)
    return n.value


def ttt_layer_backward_mse_workspace_bytes(shape: InplaceShape, dtype: torch.dtype, saved_states=False) -> int:
    return ttt_layer_backward_workspace_bytes(shape, dtype, saved_states, "mse")


def ttt_layer_backward_mse(H, X0, W_gate, W_up, W_down0, W_target, conv_w, dO, chunk: int, eta: float,
                           W_states=None, grads=None, workspace=None, doc_starts=None, update_mask=None,
                           conv_forward=False):
    """ttt_layer_backward for the MSE objective (see there)."""
    return ttt_layer_backward(H, X0, W_gate, W_up, W_down0, W_target, conv_w, dO, chunk, eta, W_states, grads,
                              workspace, doc_starts, mode="mse", update_mask=update_mask, conv_forward=conv_forward)


def ttt_layer_backward(H, X0, W_gate, W_up, W_down0, W_target, conv_w, dO, chunk: int, eta: float, W_states=None,
                       grads=None, workspace=None, doc_starts=None, mode="dot", update_mask=None, conv_forward=False,
                       W_init=None, x0_halo=None):
    """Gradients of the layer (objective `mode`, "dot" or "mse") with respect to every input, given
    dO = dLoss/dO [B, n, d], with the per-chunk states W_states kept by the forward call or recomputed (None), and
    doc_starts [B, n // chunk], update_mask [B, n // chunk], conv_forward and the resumed rows' W_init [B, d, f]
    fp32 and x0_halo [B, K-1, d] as the forward layer took them (all but the first through ttt_layer_backward_ex).
    Returns (dH, dX0, dW_gate, dW_up, dW_down0, dW_target, dconv_w): activations in the inputs' dtype, weight
    gradients fp32 summed over the batch rows; with W_init or x0_halo given, dW_init [B, d, f] fp32 and dx0_halo
    [B, K-1, d] follow (None for the one not given)."""
    if mode not in ("dot", "mse"):
        raise ValueError(f"mode must be 'dot' or 'mse', got {mode!r}")
    B, n, d = H.shape
    f = W_gate.shape[0]
    K = conv_w.shape[1]
    dt, dev = H.dtype, H.device
    for name, t, shp in (("H", H, (B, n, d)), ("X0", X0, (B, n, d)), ("W_gate", W_gate, (f, d)),
                         ("W_up", W_up, (f, d)), ("W_down0", W_down0, (d, f)), ("W_target", W_target, (d, d)),
                         ("conv_w", conv_w, (d, K)), ("dO", dO, (B, n, d))):
        _need(t, name, shp, dt, dev)
    shapes = (((B, n, d), dt), ((B, n, d), dt), ((f, d), torch.float32), ((f, d), torch.float32),
              ((d, f), torch.float32), ((d, d), torch.float32), ((d, K), torch.float32))
    if grads is None:
        grads = tuple(torch.empty(*shp, dtype=t, device=dev) for shp, t in shapes)
    for g, (shp, t) in zip(grads, shapes):
        _need(g, "gradient", shp, t, dev)
    if W_states is not None:
        _need(W_states, "W_states", (B, n // chunk, d, f), dt, dev)
    resumed = W_init is not None or x0_halo is not None
    dW_init = dx0_halo = None
    if W_init is not None:
        _need(W_init, "W_init", (B, d, f), torch.float32, dev)
        dW_init = torch.empty(B, d, f, dtype=torch.float32, device=dev)
    if x0_halo is not None:
        _need(x0_halo, "x0_halo", (B, K - 1, d), dt, dev)
        dx0_halo = torch.empty(B, K - 1, d, dtype=dt, device=dev)
    shape = _inplace_shape(B, n, d, f, chunk, K)
    nbytes = ttt_layer_backward_workspace_bytes(shape, dt, W_states is not None, mode)
    ws = _workspace(nbytes, dev, workspace)
    sp = _vp(W_states)
    doc_starts = _flags(doc_starts, "doc_starts", (B, n // chunk if chunk > 0 else 0), dev)
    dp = _vp(doc_starts)
    if update_mask is not None or conv_forward or resumed:
        um = _flags(update_mask, "update_mask", (B, n // chunk if chunk > 0 else 0), dev)
        halo_ok = x0_halo is not None and K > 1
        opts = BackwardOptions(sp, dp, _vp(um), 1 if conv_forward else 0, _vp(W_init),
                               _vp(x0_halo) if halo_ok else None, _vp(dW_init), _vp(dx0_halo) if halo_ok else None)
        _check(lib().ttt_layer_backward_ex(ctypes.byref(shape), _dt(dt), _mode(mode), float(eta), _ptr(H), _ptr(X0),
                                           _ptr(W_gate), _ptr(W_up), _ptr(W_down0), _ptr(W_target), _ptr(conv_w),
                                           _ptr(dO), ctypes.byref(opts), *[_ptr(g) for g in grads], _ptr(ws),
                                           nbytes, _stream(dev)), "ttt_layer_backward_ex")
        return tuple(grads) + (dW_init, dx0_halo) if resumed else grads
    name = "ttt_layer_backward_mse" if mode == "mse" else "ttt_layer_backward"
    _check(getattr(lib(), name)(ctypes.byref(shape), _dt(dt), float(eta), _ptr(H), _ptr(X0), _ptr(W_gate),
                                _ptr(W_up), _ptr(W_down0), _ptr(W_target), _ptr(conv_w), _ptr(dO), sp, dp,
                                *[_ptr(g) for g in grads], _ptr(ws), nbytes, _stream(dev)), name)
    return grads


def ttt_produce_z(H, W_gate, W_up, Z=None, Zt=None, with_z=True):
    """Z = silu(H W_gate^T) * (H W_up^T).  Returns (Z [B, n, f] or None, Zt [B, f, n])."""
    B, n, d = H.shape
    f = W_gate.shape[0]
    dt, dev = H.dtype, H.device
    _need(H, "H", (B, n, d), dt, dev)
    _need(W_gate, "W_gate", (f, d), dt, dev)
    _need(W_up, "W_up", (f, d), dt, dev)
    if with_z:
        Z = torch.empty(B, n, f, dtype=dt, device=dev) if Z is None else Z
        _need(Z, "Z", (B, n, f), dt, dev)
    Zt = torch.empty(B, f, n, dtype=dt, device=dev) if Zt is None else Zt
    _need(Zt, "Zt", (B, f, n), dt, dev)
    shape = _inplace_shape(B, n, d, f, max(n, 8), 1)
    _check(lib().ttt_produce_z(ctypes.byref(shape), _dt(dt), _ptr(H), _ptr(W_gate), _ptr(W_up),
                               _ptr(Z) if with_z else None, _ptr(Zt), _stream(dev)), "ttt_produce_z")
    return (Z if with_z else None), Zt


def ttt_vhat_workspace_bytes(shape: InplaceShape, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_vhat_workspace_bytes(ctypes.byref(shape), _dt(dtype), ctypes.byref(out)),
           "ttt_vhat_workspace_bytes")
    return out.value


def ttt_produce_vhat(X0, conv_w, W_target, Vt=None, workspace=None, scale: float = 1.0):
    """Vt [B, d, n] = scale * (CausalDepthwiseConv1D(X0) W_target)^T."""
    B, n, d = X0.shape
    K = conv_w.shape[1]
    dt, dev = X0.dtype, X0.device
    _need(X0, "X0", (B, n, d), dt, dev)
    _need(conv_w, "conv_w", (d, K), dt, dev)
    _need(W_target, "W_target", (d, d), dt, dev)
    Vt = torch.empty(B, d, n, dtype=dt, device=dev) if Vt is None else Vt
    _need(Vt, "Vt", (B, d, n), dt, dev)
    shape = _inplace_shape(B, n, d, 8, max(n, 8), K)
    nbytes = ttt_vhat_workspace_bytes(shape, dt)
    ws = _workspace(nbytes, dev, workspace)
    _check(lib().ttt_produce_vhat(ctypes.byref(shape), _dt(dt), float(scale), _ptr(X0), _ptr(conv_w), _ptr(W_target),
                                  _ptr(Vt), _ptr(ws), nbytes, _stream(dev)), "ttt_produce_vhat")
    return Vt


def ttt_chunk_delta(Zt, Vt, chunk: int, dW=None):
    """dW [B, k, d, f] fp32, dW[b, c] = Vhat_c^T Z_c, from Zt [B, f, n] and Vt [B, d, n]."""
    B, f, n = Zt.shape
    d = Vt.shape[1]
    dt, dev = Zt.dtype, Zt.device
    _need(Zt, "Zt", (B, f, n), dt, dev)
    _need(Vt, "Vt", (B, d, n), dt, dev)
    k = n // chunk if chunk > 0 else 0
    dW = torch.empty(B, k, d, f, dtype=torch.float32, device=dev) if dW is None else dW
    _need(dW, "dW", (B, k, d, f), torch.float32, dev)
    shape = _inplace_shape(B, n, d, f, chunk, 1)
    _check(lib().ttt_chunk_delta(ctypes.byref(shape), _dt(dt), _ptr(Zt), _ptr(Vt), _ptr(dW), _stream(dev)),
           "ttt_chunk_delta")
    return dW


def ttt_chunk_scan(dW, W_down0, eta: float, chunk: int, seq_len: int, Wc=None, W_final=None):
    """Exclusive prefix over chunks.  Returns (Wc [B, k, d, f] dtype, W_final [B, d, f] fp32)."""
    B, k, d, f = dW.shape
    dt, dev = W_down0.dtype, W_down0.device
    _need(dW, "dW", (B, k, d, f), torch.float32, dev)
    _need(W_down0, "W_down0", (d, f), dt, dev)
    Wc = torch.empty(B, k, d, f, dtype=dt, device=dev) if Wc is None else Wc
    W_final = torch.empty(B, d, f, dtype=torch.float32, device=dev) if W_final is None else W_final
    _need(Wc, "Wc", (B, k, d, f), dt, dev)
    _need(W_final, "W_final", (B, d, f), torch.float32, dev)
    if seq_len != k * chunk:
        raise ValueError("seq_len must equal k * chunk")
    shape = _inplace_shape(B, seq_len, d, f, chunk, 1)
    _check(lib().ttt_chunk_scan(ctypes.byref(shape), _dt(dt), float(eta), _ptr(W_down0), _ptr(dW), _ptr(Wc),
                                _ptr(W_final), _stream(dev)), "ttt_chunk_scan")
    return Wc, W_final


def ttt_update_scan_workspace_bytes(shape: InplaceShape, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_update_scan_workspace_bytes(ctypes.byref(shape), _dt(dtype), ctypes.byref(out)),
           "ttt_update_scan_workspace_bytes")
    return out.value


def ttt_chunk_update_scan(Zt, Vt, W_down0, chunk: int, Wc=None, W_final=None, workspace=None):
    """Fused deltas + prefix from Zt [B, f, n] and the eta-scaled target Vt [B, d, n] (ttt_produce_vhat with
    scale = eta).  Returns (Wc [B, k, d, f] dtype, W_final fp32)."""
    B, f, n = Zt.shape
    d = Vt.shape[1]
    dt, dev = Zt.dtype, Zt.device
    _need(Zt, "Zt", (B, f, n), dt, dev)
    _need(Vt, "Vt", (B, d, n), dt, dev)
    _need(W_down0, "W_down0", (d, f), dt, dev)
    k = n // chunk if chunk > 0 else 0
    Wc = torch.empty(B, k, d, f, dtype=dt, device=dev) if Wc is None else Wc
    W_final = torch.empty(B, d, f, dtype=torch.float32, device=dev) if W_final is None else W_final
    _need(Wc, "Wc", (B, k, d, f), dt, dev)
    _need(W_final, "W_final", (B, d, f), torch.float32, dev)
    shape = _inplace_shape(B, n, d, f, chunk, 1)
    need = ttt_update_scan_workspace_bytes(shape, dt) if B * n > 0 else 0
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ttt_chunk_update_scan(ctypes.byref(shape), _dt(dt), _ptr(W_down0), _ptr(Zt), _ptr(Vt), _ptr(Wc),
                                       _ptr(W_final), _ptr(workspace), wsb, _stream(dev)), "ttt_chunk_update_scan")
    return Wc, W_final


def ttt_chunk_apply(Zt, Wc, chunk: int, O=None):
    """O [B, n, d], O_c = Z_c Wc[b, c]^T, with Z given as its token-contiguous copy Zt [B, f, n]."""
    B, f, n = Zt.shape
    k, d = Wc.shape[1], Wc.shape[2]
    dt, dev = Zt.dtype, Zt.device
    _need(Zt, "Zt", (B, f, n), dt, dev)
    _need(Wc, "Wc", (B, k, d, f), dt, dev)
    if k * chunk != n:
        raise ValueError("Wc must hold one state per chunk")
    O = torch.empty(B, n, d, dtype=dt, device=dev) if O is None else O
    _need(O, "O", (B, n, d), dt, dev)
    shape = _inplace_shape(B, n, d, f, chunk, 1)
    _check(lib().ttt_chunk_apply(ctypes.byref(shape), _dt(dt), _ptr(Zt), _ptr(Wc), _ptr(O), _stream(dev)),
           "ttt_chunk_apply")
    return O


def ttt_lact_workspace_bytes(shape: LactShape, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_lact_workspace_bytes(ctypes.byref(shape), _dt(dtype), ctypes.byref(out)),
           "ttt_lact_workspace_bytes")
    return out.value


def _host_flags(update_mask, n, chunk):
    """A per-chunk host flag sequence as a ctypes uint8 array (kept alive by the caller), or None."""
    if update_mask is None:
        return None
    flags = [1 if bool(x) else 0 for x in (update_mask.tolist() if hasattr(update_mask, "tolist") else update_mask)]
    if chunk <= 0 or len(flags) != n // chunk:
        raise ValueError(f"update_mask needs {n // chunk if chunk > 0 else 0} entries, got {len(flags)}")
    return (ctypes.c_ubyte * max(1, len(flags)))(*flags)


def ttt_lact_swiglu(q, k, v, W1, W3, W2, chunk: int, eta: float, order="update_then_apply", O=None, finals=None,
                    workspace=None, update_mask=None, eta_tok=None, loss="mse", weight_norm=False, muon=False,
                    side=None, W_states=None):
    """LaCT SwiGLU layer.  Returns (O [B, H, n, dh], W1_f, W3_f [B, H, m, dh], W2_f [B, H, dh, m]).

    Options (ttt_lact_swiglu_ex): update_mask, a host sequence of n // chunk flags (only the flagged chunks
    take the update step, every chunk is applied); eta_tok, per-token learning rates [B, H, n] fp32 on the
    device; loss, "mse" or "dot"; weight_norm, L2-normalise the weight rows after every update; muon, step
    along Muon(g) (Newton-Schulz orthogonalised gradients); side, a LactSideStream on the tensors' device to run
    half of the (batch, head) rows on (None: one chain on the current stream); W_states, a [n // chunk + 1, B, H, 3,
    m * dh] tensor of the layer's dtype that receives every chunk's state for ttt_lact_swiglu_backward."""
    B, Hh, n, dh = q.shape
    m = W1.shape[1]
    dt, dev = q.dtype, q.device
    for name, t, shp in (("q", q, (B, Hh, n, dh)), ("k", k, (B, Hh, n, dh)), ("v", v, (B, Hh, n, dh)),
                         ("W1", W1, (Hh, m, dh)), ("W3", W3, (Hh, m, dh)), ("W2", W2, (Hh, dh, m))):
        _need(t, name, shp, dt, dev)
    O = torch.empty(B, Hh, n, dh, dtype=dt, device=dev) if O is None else O
    _need(O, "O", (B, Hh, n, dh), dt, dev)
    if finals is None:
        finals = (torch.empty(B, Hh, m, dh, dtype=torch.float32, device=dev),
                  torch.empty(B, Hh, m, dh, dtype=torch.float32, device=dev),
                  torch.empty(B, Hh, dh, m, dtype=torch.float32, device=dev))
    W1f, W3f, W2f = finals
    _need(W1f, "W1_f", (B, Hh, m, dh), torch.float32, dev)
    _need(W3f, "W3_f", (B, Hh, m, dh), torch.float32, dev)
    _need(W2f, "W2_f", (B, Hh, dh, m), torch.float32, dev)
    shape = LactShape(B, Hh, n, dh, m, int(chunk))
    nbytes = ttt_lact_workspace_bytes(shape, dt)
    ws = _workspace(nbytes, dev, workspace)
    ordc = _ORDERS[order] if isinstance(order, str) else int(order)
    if side is not None and side.device != dev:
        raise ValueError(f"the side stream is on {side.device}, the tensors on {dev}")
    if W_states is not None:
        _need(W_states, "W_states", (n // chunk + 1, B, Hh, 3, m * dh), dt, dev)
    if (update_mask is None and eta_tok is None and loss == "mse" and not weight_norm and not muon and side is None
            and W_states is None):
        _check(lib().ttt_lact_swiglu(ctypes.byref(shape), _dt(dt), ordc, float(eta), _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(W1), _ptr(W3), _ptr(W2), _ptr(O), _ptr(W1f), _ptr(W3f), _ptr(W2f),
                                     _ptr(ws), nbytes, _stream(dev)), "ttt_lact_swiglu")
        return O, W1f, W3f, W2f
    mask = _host_flags(update_mask, n, chunk)
    if eta_tok is not None:
        _need(eta_tok, "eta_tok", (B, Hh, n), torch.float32, dev)
    if loss not in ("mse", "dot"):
        raise ValueError(f"loss must be 'mse' or 'dot', got {loss!r}")
    opts = LactOptions(ordc, ctypes.cast(mask, ctypes.c_void_p) if mask is not None else None,
                       ctypes.c_void_p(eta_tok.data_ptr()) if eta_tok is not None and eta_tok.numel() else None,
                       1 if loss == "dot" else 0, 1 if weight_norm else 0, 1 if muon else 0,
                       *(side.handles() if side is not None else (None, None, None)), _vp(W_states))
    _check(lib().ttt_lact_swiglu_ex(ctypes.byref(shape), _dt(dt), float(eta), _ptr(q), _ptr(k), _ptr(v), _ptr(W1),
                                    _ptr(W3), _ptr(W2), ctypes.byref(opts), _ptr(O), _ptr(W1f), _ptr(W3f),
                                    _ptr(W2f), _ptr(ws), nbytes, _stream(dev)),
           "ttt_lact_swiglu_ex")
    return O, W1f, W3f, W2f


def ttt_lact_backward_workspace_bytes(shape: LactShape, dtype: torch.dtype, saved_states=False) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_lact_backward_workspace_bytes_ex(ctypes.byref(shape), _dt(dtype), int(bool(saved_states)),
                                                      ctypes.byref(out)), "ttt_lact_backward_workspace_bytes_ex")
    return out.value


def ttt_lact_swiglu_backward(q, k, v, W1, W3, W2, dO, chunk: int, eta: float, order="update_then_apply",
                             grads=None, workspace=None, update_mask=None, W_states=None):
    """Backward of the LaCT layer (squared error, plain GD) given dO = dLoss/dO [B, H, n, dh]; update_mask, a host
    sequence of n // chunk flags as the forward layer took it, and W_states, the states the forward call kept
    (both through ttt_lact_swiglu_backward_ex).  Returns (dq, dk, dv [B, H, n, dh] in the inputs' dtype, dW1, dW3
    [H, m, dh], dW2 [H, dh, m] fp32, summed over the batch rows)."""
    B, Hh, n, dh = q.shape
    m = W1.shape[1]
    dt, dev = q.dtype, q.device
    for name, t, shp in (("q", q, (B, Hh, n, dh)), ("k", k, (B, Hh, n, dh)), ("v", v, (B, Hh, n, dh)),
                         ("W1", W1, (Hh, m, dh)), ("W3", W3, (Hh, m, dh)), ("W2", W2, (Hh, dh, m)),
                         ("dO", dO, (B, Hh, n, dh))):
        _need(t, name, shp, dt, dev)
    shapes = (((B, Hh, n, dh), dt),) * 3 + (((Hh, m, dh), torch.float32), ((Hh, m, dh), torch.float32),
                                            ((Hh, dh, m), torch.float32))
    if grads is None:
        grads = tuple(torch.empty(*shp, dtype=t, device=dev) for shp, t in shapes)
    for gt, (shp, t) in zip(grads, shapes):
        _need(gt, "gradient", shp, t, dev)
    shape = LactShape(B, Hh, n, dh, m, int(chunk))
    if W_states is not None:
        _need(W_states, "W_states", (n // chunk + 1, B, Hh, 3, m * dh), dt, dev)
    nbytes = ttt_lact_backward_workspace_bytes(shape, dt, W_states is not None)
    ws = _workspace(nbytes, dev, workspace)
    ordc = _ORDERS[order] if isinstance(order, str) else int(order)
    if update_mask is not None or W_states is not None:
        mask = _host_flags(update_mask, n, chunk)
        opts = LactOptions(ordc, ctypes.cast(mask, ctypes.c_void_p) if mask is not None else None, None, 0, 0, 0,
                           None, None, None, _vp(W_states))
        _check(lib().ttt_lact_swiglu_backward_ex(ctypes.byref(shape), _dt(dt), float(eta), _ptr(q), _ptr(k),
                                                 _ptr(v), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(dO), ctypes.byref(opts),
                                                 *[_ptr(g) for g in grads], _ptr(ws), nbytes, _stream(dev)),
               "ttt_lact_swiglu_backward_ex")
        return grads
    _check(lib().ttt_lact_swiglu_backward(ctypes.byref(shape), _dt(dt), ordc, float(eta), _ptr(q), _ptr(k), _ptr(v),
                                          _ptr(W1), _ptr(W3), _ptr(W2), _ptr(dO), *[_ptr(g) for g in grads],
                                          _ptr(ws), nbytes, _stream(dev)), "ttt_lact_swiglu_backward")
    return grads


# ---------------------------------------------------------------------------------- gated delta rule, layer norm
#
# What follows from shapes, strides and types alone (checks, the C structs, workspace sizes) is made once for each
# combination and kept; a call looks it up, checks devices and addresses, allocates and launches.


def _launch(device: torch.device, what: str, fn, *args):
    """Calls a C entry on the tensors' device and its current stream."""
    if device.index == torch.cuda.current_device():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if status != TTT_OK:
        raise TTTError(status, what)


def _at(t):
    """A tensor's address, or None for a missing or empty one."""
    return (t.data_ptr() or None) if t is not None else None


def _meta(t, name, device, aligned=True):
    """A tensor's shape, strides and type, its kind, device and (rows') address checked."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (the layer runs only in the HIP library)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if aligned and t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    return t.shape, t.stride(), t.dtype


def _strides(meta, name, shape, dtype, rows=True, out=False) -> DeltaStrides:
    """Checks a [B, H, n, d] (or, with rows=False, a [B, H, n]) tensor of any batch, head and token strides, and
    gives them.  Outputs must not hold two elements at one place."""
    size, st, dt = meta
    if size != shape:
        raise ValueError(f"{name} has shape {tuple(size)}, expected {shape}")
    if dt != dtype:
        raise TypeError(f"{name} has dtype {dt}, expected {dtype}")
    if 0 not in shape:
        if rows and (st[3] != 1 and shape[3] > 1 or any(s * dtype.itemsize % 16 for s, n in zip(st[:3], shape) if n > 1)):
            raise ValueError(f"{name}'s last index must be contiguous and its rows 16-byte aligned (strides {st})")
        reach = 1
        for s, n in sorted((s, n) for s, n in zip(st, shape) if n > 1):
            if out and s < reach:
                raise ValueError(f"{name} is written and must not overlap itself (strides {st})")
            reach = s * n
    return DeltaStrides(*(s if n > 1 else 0 for s, n in zip(st[:3], shape)))


@functools.lru_cache(maxsize=256)
def _delta_plan(q, k, v, g, beta, O, num):
    """(byref of DeltaShape, its dtype code, DeltaLayout, workspace bytes, states' rows) of a forward call."""
    shape, strides = _delta_strides(q, k, v, g, beta)
    layout = DeltaLayout(*strides, _strides(O, "O", tuple(v[0]), q[2], out=True))
    return (ctypes.byref(shape), _dt(q[2]), layout, ttt_gated_delta_workspace_bytes(shape, q[2], num),
            (shape.batch if num < 0 else num, shape.v_heads, shape.v_dim, shape.k_dim))


def _delta_strides(q, k, v, g, beta):
    if len(q[0]) != 4 or len(v[0]) != 4:
        raise ValueError(f"q and v are [B, H, n, d], got {tuple(q[0])} and {tuple(v[0])}")
    (B, Hk, n, dk), Hv, dv, dt = q[0], v[0][1], v[0][3], q[2]
    return DeltaShape(B, n, Hk, Hv, dk, dv), (
        _strides(q, "q", (B, Hk, n, dk), dt), _strides(k, "k", (B, Hk, n, dk), dt), _strides(v, "v", (B, Hv, n, dv), dt),
        _strides(g, "g", (B, Hv, n), torch.float32, rows=False),
        _strides(beta, "beta", (B, Hv, n), torch.float32, rows=False))


def _delta_metas(q, k, v, g, beta, dev):
    return (_meta(q, "q", dev), _meta(k, "k", dev), _meta(v, "v", dev), _meta(g, "g", dev, False),
            _meta(beta, "beta", dev, False))


def _seq_starts(seq_starts, B, device):
    """Checks packed rows' starts [sequences + 1] (int32, device); the number of sequences, or -1."""
    if seq_starts is None:
        return -1
    if not isinstance(seq_starts, torch.Tensor) or seq_starts.dim() != 1 or seq_starts.numel() < 1:
        raise ValueError("seq_starts must be a tensor [sequences + 1]")
    _need(seq_starts, "seq_starts", seq_starts.shape, torch.int32, device)
    if B != 1:
        raise ValueError(f"packed sequences lie in one batch row, got {B}")
    return seq_starts.numel() - 1


def ttt_gated_delta_workspace_bytes(shape: DeltaShape, dtype: torch.dtype, num_seqs: int = -1) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_gated_delta_workspace_bytes(ctypes.byref(shape), _dt(dtype), int(num_seqs), ctypes.byref(out)),
           "ttt_gated_delta_workspace_bytes")
    return out.value


def ttt_gated_delta(q, k, v, g, beta, scale=None, W_init=None, seq_starts=None, O=None, W_final=None,
                    workspace=None):
    """The gated delta rule over whole sequences: per value head W_t = exp(g_t) W_{t-1} + beta_t (v_t -
    exp(g_t) W_{t-1} k_t) k_t^T, o_t = scale W_t q_t.  Returns (O [B, Hv, n, dv], W_final [sequences, Hv, dv, dk]
    fp32).

    q, k [B, Hk, n, dk] and v [B, Hv, n, dv] share a dtype, g and beta [B, Hv, n] are fp32; each may have any
    batch, head and token strides (a token-major tensor's transpose(1, 2)), and O, if not given, is laid out like
    v.  Hv is a multiple of Hk: value head h reads key head h // (Hv // Hk).  scale: dk ** -0.5 if None.
    W_init [sequences, Hv, dv, dk] fp32: the states to start from (zero if None).  seq_starts, an int32 device
    tensor [sequences + 1]: packed sequences of any lengths in one batch row; tokens behind the last of them are
    not read and their rows of O are left as they are."""
    dev = q.device
    metas = _delta_metas(q, k, v, g, beta, dev)
    num = _seq_starts(seq_starts, q.shape[0], dev)
    O = torch.empty_like(v) if O is None else O
    shape, dt, layout, nbytes, states = _delta_plan(*metas, _meta(O, "O", dev), num)
    if W_init is not None:
        _need(W_init, "W_init", states, torch.float32, dev)
    W_final = torch.empty(states, dtype=torch.float32, device=dev) if W_final is None else W_final
    _need(W_final, "W_final", states, torch.float32, dev)
    ws = _workspace(nbytes, dev, workspace)
    opts = DeltaOptions(_at(W_init), _at(seq_starts), max(num, 0), ctypes.pointer(layout))
    _launch(dev, "ttt_gated_delta", lib().ttt_gated_delta, shape, dt,
            states[3] ** -0.5 if scale is None else float(scale), _at(q), _at(k), _at(v), _at(g), _at(beta),
            ctypes.byref(opts), _at(O), _at(W_final), _at(ws), nbytes)
    return O, W_final


def ttt_gated_delta_backward_workspace_bytes(shape: DeltaShape, dtype: torch.dtype, num_seqs: int = -1) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_gated_delta_backward_workspace_bytes(ctypes.byref(shape), _dt(dtype), int(num_seqs),
                                                          ctypes.byref(out)),
           "ttt_gated_delta_backward_workspace_bytes")
    return out.value


@functools.lru_cache(maxsize=256)
def _delta_backward_plan(q, k, v, g, beta, dO, dq, dk, dv, dg, dbeta, gate, num):
    shape, strides = _delta_strides(q, k, v, g, beta)
    qs, vs, gs, dt = tuple(q[0]), tuple(v[0]), tuple(g[0]), q[2]
    grads = DeltaGradLayout(_strides(dO, "dO", vs, dt), _strides(dq, "dq", qs, dt, out=True),
                            _strides(dk, "dk", qs, dt, out=True), _strides(dv, "dv", vs, dt, out=True),
                            _strides(dg, "dg", gs, gate, rows=False, out=True),
                            _strides(dbeta, "dbeta", gs, gate, rows=False, out=True), gate == torch.float32)
    return (ctypes.byref(shape), _dt(dt), DeltaLayout(*strides, DeltaStrides()), grads,
            ttt_gated_delta_backward_workspace_bytes(shape, dt, num),
            (shape.batch if num < 0 else num, shape.v_heads, shape.v_dim, shape.k_dim))


def ttt_gated_delta_backward(q, k, v, g, beta, dO, dW_final=None, scale=None, W_init=None, seq_starts=None, dq=None,
                             dk=None, dv=None, dg=None, dbeta=None, dW_init=None, workspace=None, gate_dtype=None):
    """Backward of ttt_gated_delta from its inputs (the states are made again), dO = dLoss/dO [B, Hv, n, dv] and, where
    the loss depends on the final states too, dW_final [sequences, Hv, dv, dk] fp32.  Returns (dq, dk, dv, dg, dbeta)
    in q's dtype, each laid out like its input if not given, and dW_init [sequences, Hv, dv, dk] fp32 (None without
    W_init, unless given).  gate_dtype: the dtype of dg and dbeta, torch.float32 (as g and beta are; the sums as they
    are made) or q's (None: rounded once).  dO and the gradients may have any strides that the inputs may; rows of tokens
    that belong to no sequence are left as they are."""
    dev, t = q.device, q.dtype
    gate = t if gate_dtype is None else gate_dtype
    if gate not in (t, torch.float32):
        raise TypeError(f"gate_dtype must be float32 or {t}, got {gate}")
    metas = _delta_metas(q, k, v, g, beta, dev)
    num = _seq_starts(seq_starts, q.shape[0], dev)
    dq, dk, dv = (torch.empty_like(x) if d is None else d for d, x in ((dq, q), (dk, k), (dv, v)))
    dg, dbeta = (torch.empty_like(x, dtype=gate) if d is None else d for d, x in ((dg, g), (dbeta, beta)))
    shape, dt, layout, grads, nbytes, states = _delta_backward_plan(
        *metas, _meta(dO, "dO", dev), _meta(dq, "dq", dev), _meta(dk, "dk", dev), _meta(dv, "dv", dev),
        _meta(dg, "dg", dev, False), _meta(dbeta, "dbeta", dev, False), gate, num)
    if W_init is not None and dW_init is None:
        dW_init = torch.empty_like(W_init)
    for d, name in ((W_init, "W_init"), (dW_final, "dW_final"), (dW_init, "dW_init")):
        if d is not None:
            _need(d, name, states, torch.float32, dev)
    ws = _workspace(nbytes, dev, workspace)
    opts = DeltaOptions(_at(W_init), _at(seq_starts), max(num, 0), ctypes.pointer(layout))
    _launch(dev, "ttt_gated_delta_backward", lib().ttt_gated_delta_backward, shape, dt,
            states[3] ** -0.5 if scale is None else float(scale), _at(q), _at(k), _at(v), _at(g), _at(beta), _at(dO),
            _at(dW_final), ctypes.byref(opts), ctypes.byref(grads), _at(dq), _at(dk), _at(dv), _at(dg), _at(dbeta),
            _at(dW_init), _at(ws), nbytes)
    return dq, dk, dv, dg, dbeta, dW_init


@functools.lru_cache(maxsize=256)
def _step_shape(*sizes):
    return ctypes.byref(DeltaStepShape(*sizes))


def ttt_gated_delta_step(q, k, v, g, beta, W, slots=None, scale=None, O=None):
    """One token of the gated delta rule for each row of a serving batch.  q, k [rows, Hk, dk], v [rows, Hv, dv] of
    one dtype, g, beta [rows, Hv] fp32; W [states, Hv, dv, dk] fp32 is the pool of states, updated in place; slots
    [rows] int32 on the device names each row's state (a slot outside the pool, such as -1: a padding row, whose
    output is zero; rows of one slot go in row order; at most 65536 rows; None: row r's state is W[r]).  Returns O
    [rows, Hv, dv]."""
    (R, Hk, dk), (_, Hv, dv), P = q.shape, v.shape, W.shape[0]
    dt, dev = q.dtype, q.device
    _need(q, "q", (R, Hk, dk), dt, dev)
    _need(k, "k", (R, Hk, dk), dt, dev)
    _need(v, "v", (R, Hv, dv), dt, dev)
    _need(g, "g", (R, Hv), torch.float32, dev)
    _need(beta, "beta", (R, Hv), torch.float32, dev)
    _need(W, "W", (P, Hv, dv, dk), torch.float32, dev)
    if slots is not None:
        _need(slots, "slots", (R,), torch.int32, dev)
    if O is None:
        O = torch.empty_like(v)
    else:
        _need(O, "O", (R, Hv, dv), dt, dev)
    _launch(dev, "ttt_gated_delta_step", lib().ttt_gated_delta_step, _step_shape(R, P, Hk, Hv, dk, dv), _dt(dt),
            dk ** -0.5 if scale is None else float(scale), _at(q), _at(k), _at(v), _at(g), _at(beta), _at(W), _at(slots),
            _at(O))
    return O


def _norm_vector(t, name, d, dt, dev):
    if t is not None:
        _need(t, name, (d,), dt, dev)


def ttt_layer_norm(x, weight=None, bias=None, eps=1e-5, Y=None, mean=None, rstd=None):
    """Layer norm over the last index of x [..., d] (contiguous): returns (Y like x, mean [...], rstd [...] fp32).
    weight and bias [d] of x's dtype, or None."""
    shape, dt, dev = x.shape, x.dtype, x.device
    d, lead = shape[-1], shape[:-1]
    _need(x, "x", shape, dt, dev)
    _norm_vector(weight, "weight", d, dt, dev)
    _norm_vector(bias, "bias", d, dt, dev)
    Y = torch.empty_like(x) if Y is None else Y
    mean = torch.empty(lead, dtype=torch.float32, device=dev) if mean is None else mean
    rstd = torch.empty(lead, dtype=torch.float32, device=dev) if rstd is None else rstd
    _need(Y, "Y", shape, dt, dev)
    _need(mean, "mean", lead, torch.float32, dev)
    _need(rstd, "rstd", lead, torch.float32, dev)
    _launch(dev, "ttt_layer_norm", lib().ttt_layer_norm, mean.numel(), d, _dt(dt), float(eps), _at(x), _at(weight),
            _at(bias), _at(Y), _at(mean), _at(rstd))
    return Y, mean, rstd


@functools.lru_cache(maxsize=256)
def ttt_layer_norm_backward_workspace_bytes(rows: int, dim: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_layer_norm_backward_workspace_bytes(int(rows), int(dim), _dt(dtype), ctypes.byref(out)),
           "ttt_layer_norm_backward_workspace_bytes")
    return out.value


def ttt_layer_norm_backward(x, weight, dY, mean, rstd, bias=True, dx=None, dweight=None, dbias=None,
                            workspace=None):
    """Backward of ttt_layer_norm given its mean and rstd.  Returns (dx like x, dweight [d] fp32 or None where
    weight is None, dbias [d] fp32 or None with bias=False)."""
    shape, dt, dev = x.shape, x.dtype, x.device
    d, lead = shape[-1], shape[:-1]
    _need(x, "x", shape, dt, dev)
    _need(dY, "dY", shape, dt, dev)
    _norm_vector(weight, "weight", d, dt, dev)
    _need(mean, "mean", lead, torch.float32, dev)
    _need(rstd, "rstd", lead, torch.float32, dev)
    dx = torch.empty_like(x) if dx is None else dx
    _need(dx, "dx", shape, dt, dev)
    if weight is not None and dweight is None:
        dweight = torch.empty(d, dtype=torch.float32, device=dev)
    if bias and dbias is None:
        dbias = torch.empty(d, dtype=torch.float32, device=dev)
    _norm_vector(dweight, "dweight", d, torch.float32, dev)
    _norm_vector(dbias, "dbias", d, torch.float32, dev)
    rows = mean.numel()
    nbytes = ttt_layer_norm_backward_workspace_bytes(rows, d, dt)
    ws = _workspace(nbytes, dev, workspace)
    _launch(dev, "ttt_layer_norm_backward", lib().ttt_layer_norm_backward, rows, d, _dt(dt), _at(x), _at(weight), _at(dY),
            _at(mean), _at(rstd), _at(dx), _at(dweight), _at(dbias), _at(ws), nbytes)
    return dx, dweight, dbias


# -------------------------------------------------- root-mean-square norm, short convolution, selective scan


def ttt_rms_norm(x, weight=None, residual=None, eps=1e-5, out_dtype=None, group=None, Y=None, H=None, rstd=None,
                 scale=None):
    """Root-mean-square norm over the last index of H = x + residual (x where residual is None), x [..., d]
    (contiguous), weight [d] of x's dtype or None.  Returns (Y, H, rstd [...] fp32, scale).

    out_dtype None: Y of x's dtype, scale None.  torch.float8_e4m3fn: Y = H rstd weight / scale in 8 bits, scale [...]
    fp32 the largest |H rstd weight| of a row over 448, or, with group 32, 64 or 128, [..., ceil(d / group)] that of
    each group of columns; at least 2^-126."""
    shape, dt, dev = x.shape, x.dtype, x.device
    d, lead = shape[-1], shape[:-1]
    _need(x, "x", shape, dt, dev)
    _norm_vector(weight, "weight", d, dt, dev)
    if residual is not None:
        _need(residual, "residual", shape, dt, dev)
        if H is None:
            H = torch.empty_like(x)
        else:
            _need(H, "H", shape, dt, dev)
    bits8 = out_dtype is not None and out_dtype != dt
    if bits8 and out_dtype != torch.float8_e4m3fn:
        raise TypeError(f"out_dtype must be {dt} or float8_e4m3fn, got {out_dtype}")
    if group is not None and (not bits8 or group not in (32, 64, 128)):
        raise ValueError(f"group must be 32, 64 or 128, and is of 8-bit outputs, got {group}")
    if Y is None:
        Y = torch.empty_like(x, dtype=out_dtype) if bits8 else torch.empty_like(x)
    else:
        _need(Y, "Y", shape, out_dtype if bits8 else dt, dev)
    if rstd is None:
        rstd = x.new_empty(lead, dtype=torch.float32)
    else:
        _need(rstd, "rstd", lead, torch.float32, dev)
    if bits8:
        scales = lead if group is None else (*lead, -(-d // group))
        if scale is None:
            scale = x.new_empty(scales, dtype=torch.float32)
        else:
            _need(scale, "scale", scales, torch.float32, dev)
    elif scale is not None:
        raise ValueError("scale is of 8-bit outputs")
    _launch(dev, "ttt_rms_norm", lib().ttt_rms_norm, rstd.numel(), d, _dt(dt), float(eps), _at(x), _at(residual),
            _at(weight), _at(H) if residual is not None else None, _at(Y), _at(rstd), _at(scale), group or 0)
    return Y, x if residual is None else H, rstd, scale


@functools.lru_cache(maxsize=256)
def ttt_rms_norm_backward_workspace_bytes(rows: int, dim: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_rms_norm_backward_workspace_bytes(int(rows), int(dim), _dt(dtype), ctypes.byref(out)),
           "ttt_rms_norm_backward_workspace_bytes")
    return out.value


def ttt_rms_norm_backward(H, weight, dY, rstd, dH=None, dx=None, dweight=None, workspace=None):
    """Backward of ttt_rms_norm (Y of x's dtype) given its H and rstd; dH, if not None, is what comes back to H from its
    other uses.  Returns (dx like H, the gradient of x and of the residual, dweight [d] fp32 or None where weight is
    None)."""
    shape, dt, dev = H.shape, H.dtype, H.device
    d, lead = shape[-1], shape[:-1]
    _need(H, "H", shape, dt, dev)
    _need(dY, "dY", shape, dt, dev)
    _norm_vector(weight, "weight", d, dt, dev)
    _need(rstd, "rstd", lead, torch.float32, dev)
    if dH is not None:
        _need(dH, "dH", shape, dt, dev)
    if dx is None:
        dx = torch.empty_like(H)
    else:
        _need(dx, "dx", shape, dt, dev)
    if dweight is not None:
        _need(dweight, "dweight", (d,), torch.float32, dev)
    elif weight is not None:
        dweight = weight.new_empty(d, dtype=torch.float32)
    rows = rstd.numel()
    nbytes = ttt_rms_norm_backward_workspace_bytes(rows, d, dt)
    ws = _workspace(nbytes, dev, workspace)
    _launch(dev, "ttt_rms_norm_backward", lib().ttt_rms_norm_backward, rows, d, _dt(dt), _at(H), _at(weight), _at(dY),
            _at(rstd), _at(dH), _at(dx), _at(dweight), _at(ws), nbytes)
    return dx, dweight


def _rows(meta, name, shape, dtype, out=False) -> RowStrides:
    """Checks a [B, n, d] tensor of any batch and token strides, and gives them.  Outputs must not hold two elements at
    one place."""
    size, st, dt = meta
    if size != shape:
        raise ValueError(f"{name} has shape {tuple(size)}, expected {shape}")
    if dt != dtype:
        raise TypeError(f"{name} has dtype {dt}, expected {dtype}")
    if 0 not in shape:
        if st[2] != 1 and shape[2] > 1:
            raise ValueError(f"{name}'s last index must be contiguous (strides {st})")
        reach = shape[2]
        for s, n in sorted((s, n) for s, n in zip(st[:2], shape) if n > 1):
            if out and s < reach:
                raise ValueError(f"{name} is written and must not overlap itself (strides {st})")
            reach = s * n
    return RowStrides(*(s if n > 1 else 0 for s, n in zip(st[:2], shape)))


def _conv_shape(x, w):
    if len(x[0]) != 3 or len(w[0]) != 2:
        raise ValueError(f"x is [B, n, d] and conv_w [d, K], got {tuple(x[0])} and {tuple(w[0])}")
    return ConvShape(*x[0], w[0][1])


@functools.lru_cache(maxsize=256)
def _conv_plan(x, w, Y, num):
    """(byref of ConvShape, its dtype code, ConvLayout, x_final's shape) of a forward call."""
    shape = _conv_shape(x, w)
    layout = ConvLayout(_rows(x, "x", tuple(x[0]), x[2]), _rows(Y, "Y", tuple(x[0]), x[2], out=True))
    return ctypes.byref(shape), _dt(x[2]), layout, (shape.batch if num < 0 else num, max(shape.taps - 1, 0), shape.dim)


def _conv_vectors(conv_w, bias, d, dt, dev):
    _need(conv_w, "conv_w", (d, conv_w.shape[-1]), dt, dev)
    _norm_vector(bias, "bias", d, dt, dev)


def ttt_short_conv(x, conv_w, bias=None, silu=True, x_init=None, seq_starts=None, Y=None, x_final=None):
    """Causal depthwise convolution over the tokens, with SiLU unless silu is False: z_t = bias + sum_j conv_w[:, j]
    x_{t-K+1+j}.  Returns (Y [B, n, d], x_final [sequences, K - 1, d], each sequence's last K - 1 rows).

    x [B, n, d] of any batch and token strides (Y, if not given, is contiguous), conv_w [d, K] (K in 1..8) and bias [d]
    of its dtype.  x_init [sequences, K - 1, d]: the rows before each sequence's first (an earlier call's x_final; zero
    if None).  seq_starts, an int32 device tensor [sequences + 1]: packed sequences in one batch row; tokens that belong
    to none are not read and their rows of Y are left as they are."""
    dev, dt = x.device, x.dtype
    _conv_vectors(conv_w, bias, x.shape[-1], dt, dev)
    num = _seq_starts(seq_starts, x.shape[0], dev)
    Y = x.new_empty(x.shape) if Y is None else Y
    shape, code, layout, halo = _conv_plan(_meta(x, "x", dev, False), _meta(conv_w, "conv_w", dev, False),
                                           _meta(Y, "Y", dev, False), num)
    if x_init is not None:
        _need(x_init, "x_init", halo, dt, dev)
    if x_final is None:
        x_final = x.new_empty(halo)
    else:
        _need(x_final, "x_final", halo, dt, dev)
    opts = ConvOptions(_at(bias), bool(silu), _at(x_init), _at(seq_starts), max(num, 0), ctypes.pointer(layout))
    _launch(dev, "ttt_short_conv", lib().ttt_short_conv, shape, code, _at(x), _at(conv_w), ctypes.byref(opts), _at(Y),
            _at(x_final))
    return Y, x_final


def ttt_short_conv_backward_workspace_bytes(shape: ConvShape, dtype: torch.dtype, num_seqs: int = -1) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_short_conv_backward_workspace_bytes(ctypes.byref(shape), _dt(dtype), int(num_seqs),
                                                         ctypes.byref(out)), "ttt_short_conv_backward_workspace_bytes")
    return out.value


@functools.lru_cache(maxsize=256)
def _conv_backward_plan(x, w, dY, dx, num):
    shape, size, dt = _conv_shape(x, w), tuple(x[0]), x[2]
    layout = ConvLayout(_rows(x, "x", size, dt), RowStrides())
    grads = ConvGradLayout(_rows(dY, "dY", size, dt), _rows(dx, "dx", size, dt, out=True))
    return (ctypes.byref(shape), _dt(dt), layout, grads, ttt_short_conv_backward_workspace_bytes(shape, dt, num),
            (shape.batch if num < 0 else num, max(shape.taps - 1, 0), shape.dim))


def ttt_short_conv_backward(x, conv_w, dY, bias=None, silu=True, x_init=None, seq_starts=None, dx_final=None, dx=None,
                            dconv_w=None, dbias=None, dx_init=None, workspace=None):
    """Backward of ttt_short_conv from its inputs, dY [B, n, d] and, where the loss depends on x_final too, dx_final.
    Returns (dx [B, n, d], dconv_w [d, K] fp32, dbias [d] fp32 (None without bias, unless given), dx_init [sequences,
    K - 1, d] (None without x_init, unless given)).  Rows of tokens that belong to no sequence are left as they are."""
    dev, dt = x.device, x.dtype
    _conv_vectors(conv_w, bias, x.shape[-1], dt, dev)
    num = _seq_starts(seq_starts, x.shape[0], dev)
    dx = x.new_empty(x.shape) if dx is None else dx
    shape, code, layout, grads, nbytes, halo = _conv_backward_plan(
        _meta(x, "x", dev, False), _meta(conv_w, "conv_w", dev, False), _meta(dY, "dY", dev, False),
        _meta(dx, "dx", dev, False), num)
    if x_init is not None and dx_init is None:
        dx_init = torch.empty(halo, dtype=dt, device=dev)
    for t, name in ((x_init, "x_init"), (dx_final, "dx_final"), (dx_init, "dx_init")):
        if t is not None:
            _need(t, name, halo, dt, dev)
    if dconv_w is None:
        dconv_w = conv_w.new_empty(conv_w.shape, dtype=torch.float32)
    else:
        _need(dconv_w, "dconv_w", conv_w.shape, torch.float32, dev)
    if dbias is not None:
        _need(dbias, "dbias", (x.shape[-1],), torch.float32, dev)
    elif bias is not None:
        dbias = bias.new_empty(bias.shape, dtype=torch.float32)
    ws = _workspace(nbytes, dev, workspace)
    opts = ConvOptions(_at(bias), bool(silu), _at(x_init), _at(seq_starts), max(num, 0), ctypes.pointer(layout))
    _launch(dev, "ttt_short_conv_backward", lib().ttt_short_conv_backward, shape, code, _at(x), _at(conv_w), _at(dY),
            _at(dx_final), ctypes.byref(opts), ctypes.byref(grads), _at(dx), _at(dconv_w), _at(dbias), _at(dx_init),
            _at(ws), nbytes)
    return dx, dconv_w, dbias, dx_init


def ttt_short_conv_step(x, conv_w, halo, bias=None, silu=True, slots=None, Y=None):
    """One token of the short convolution for each row of a serving batch.  x [rows, d], conv_w [d, K], bias [d] of one
    dtype; halo [states, K - 1, d] is the pool of earlier rows, moved on in place; slots [rows] int32 on the device
    names each row's (a slot outside the pool, such as -1: a padding row, whose output is zero; rows of one slot go in
    row order; at most 65536 rows; None: row r's is halo[r]).  Returns Y [rows, d]."""
    (R, d), (P, K1, _), dt, dev = x.shape, halo.shape, x.dtype, x.device
    _need(x, "x", (R, d), dt, dev)
    _need(conv_w, "conv_w", (d, K1 + 1), dt, dev)
    _norm_vector(bias, "bias", d, dt, dev)
    _need(halo, "halo", (P, K1, d), dt, dev)
    if slots is not None:
        _need(slots, "slots", (R,), torch.int32, dev)
    if Y is None:
        Y = torch.empty_like(x)
    else:
        _need(Y, "Y", (R, d), dt, dev)
    _launch(dev, "ttt_short_conv_step", lib().ttt_short_conv_step, R, P, d, K1 + 1, _dt(dt), bool(silu), _at(x),
            _at(conv_w), _at(bias), _at(halo), _at(slots), _at(Y))
    return Y


def _scan_heads(A, D, dt_bias, H, dev):
    _need(A, "A", (H,), torch.float32, dev)
    _norm_vector(D, "D", H, torch.float32, dev)
    _norm_vector(dt_bias, "dt_bias", H, torch.float32, dev)


def _scan_strides(x, dt, B, C):
    if len(x[0]) != 4 or len(B[0]) != 4:
        raise ValueError(f"x is [B, H, n, P] and B [B, G, n, N], got {tuple(x[0])} and {tuple(B[0])}")
    (b, H, n, P), G, N, t = x[0], B[0][1], B[0][3], x[2]
    return ScanShape(b, n, H, G, P, N), (
        _strides(x, "x", (b, H, n, P), t), _strides(dt, "dt", (b, H, n), torch.float32, rows=False),
        _strides(B, "B", (b, G, n, N), t), _strides(C, "C", (b, G, n, N), t))


def _scan_metas(x, dt, B, C, dev):
    return _meta(x, "x", dev), _meta(dt, "dt", dev, False), _meta(B, "B", dev), _meta(C, "C", dev)


def ttt_selective_scan_workspace_bytes(shape: ScanShape, dtype: torch.dtype, num_seqs: int = -1) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_selective_scan_workspace_bytes(ctypes.byref(shape), _dt(dtype), int(num_seqs), ctypes.byref(out)),
           "ttt_selective_scan_workspace_bytes")
    return out.value


@functools.lru_cache(maxsize=256)
def _scan_plan(x, dt, B, C, O, num):
    """(byref of ScanShape, its dtype code, ScanLayout, workspace bytes, states' shape) of a forward call."""
    shape, strides = _scan_strides(x, dt, B, C)
    layout = ScanLayout(*strides, _strides(O, "O", tuple(x[0]), x[2], out=True))
    return (ctypes.byref(shape), _dt(x[2]), layout, ttt_selective_scan_workspace_bytes(shape, x[2], num),
            (shape.batch if num < 0 else num, shape.heads, shape.head_dim, shape.state))


def ttt_selective_scan(x, dt, A, B, C, D=None, dt_bias=None, softplus=False, S_init=None, seq_starts=None, O=None,
                       S_final=None, workspace=None):
    """The selective scan over whole sequences: per head S_t = exp(A r_t) S_{t-1} + r_t x_t B_t^T, o_t = S_t C_t + D x_t
    with r_t = dt_t + dt_bias, or softplus of that.  Returns (O [B, H, n, P], S_final [sequences, H, P, N] fp32).

    x [B, H, n, P] and B, C [B, G, n, N] share a dtype, dt [B, H, n], A, D and dt_bias [H] are fp32, A r_t at most 0;
    tensors of tokens may have any batch, head and token strides (a token-major tensor's transpose(1, 2)), and O, if not
    given, is laid out like x.  H is a multiple of G: head h reads group h // (H // G).  S_init [sequences, H, P, N]
    fp32: the states to start from (zero if None).  seq_starts, an int32 device tensor [sequences + 1]: packed sequences
    of any lengths in one batch row; tokens that belong to none are not read and their rows of O are left as they are."""
    dev = x.device
    metas = _scan_metas(x, dt, B, C, dev)
    _scan_heads(A, D, dt_bias, x.shape[1], dev)
    num = _seq_starts(seq_starts, x.shape[0], dev)
    O = torch.empty_like(x) if O is None else O
    shape, code, layout, nbytes, states = _scan_plan(*metas, _meta(O, "O", dev), num)
    if S_init is not None:
        _need(S_init, "S_init", states, torch.float32, dev)
    if S_final is None:
        S_final = A.new_empty(states)
    else:
        _need(S_final, "S_final", states, torch.float32, dev)
    ws = _workspace(nbytes, dev, workspace) if nbytes else None
    opts = ScanOptions(_at(D), _at(dt_bias), bool(softplus), _at(S_init), _at(seq_starts), max(num, 0),
                       ctypes.pointer(layout))
    _launch(dev, "ttt_selective_scan", lib().ttt_selective_scan, shape, code, _at(x), _at(dt), _at(A), _at(B), _at(C),
            ctypes.byref(opts), _at(O), _at(S_final), _at(ws), nbytes)
    return O, S_final


def ttt_selective_scan_backward_workspace_bytes(shape: ScanShape, dtype: torch.dtype, num_seqs: int = -1) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ttt_selective_scan_backward_workspace_bytes(ctypes.byref(shape), _dt(dtype), int(num_seqs),
                                                             ctypes.byref(out)),
           "ttt_selective_scan_backward_workspace_bytes")
    return out.value


@functools.lru_cache(maxsize=256)
def _scan_backward_plan(x, dt, B, C, dO, dx, ddt, dB, dC, num):
    shape, strides = _scan_strides(x, dt, B, C)
    xs, ds, bs, t = tuple(x[0]), tuple(dt[0]), tuple(B[0]), x[2]
    grads = ScanGradLayout(_strides(dO, "dO", xs, t), _strides(dx, "dx", xs, t, out=True),
                           _strides(ddt, "ddt", ds, torch.float32, rows=False, out=True),
                           _strides(dB, "dB", bs, t, out=True), _strides(dC, "dC", bs, t, out=True))
    return (ctypes.byref(shape), _dt(t), ScanLayout(*strides, DeltaStrides()), grads,
            ttt_selective_scan_backward_workspace_bytes(shape, t, num),
            (shape.batch if num < 0 else num, shape.heads, shape.head_dim, shape.state))


def ttt_selective_scan_backward(x, dt, A, B, C, dO, D=None, dt_bias=None, softplus=False, dS_final=None, S_init=None,
                                seq_starts=None, dx=None, ddt=None, dA=None, dB=None, dC=None, dD=None, ddt_bias=None,
                                dS_init=None, workspace=None):
    """Backward of ttt_selective_scan from its inputs (the states are made again), dO = dLoss/dO [B, H, n, P] and, where
    the loss depends on the final states too, dS_final [sequences, H, P, N] fp32.  Returns (dx, ddt, dA, dB, dC, dD,
    ddt_bias, dS_init): dx, dB, dC in x's dtype, the others fp32, tensors of tokens laid out like their inputs if not
    given; dD, ddt_bias and dS_init are None without D, dt_bias and S_init, unless given.  dO and the gradients may have
    any strides that the inputs may; rows of tokens that belong to no sequence are left as they are."""
    dev, H = x.device, x.shape[1]
    metas = _scan_metas(x, dt, B, C, dev)
    _scan_heads(A, D, dt_bias, H, dev)
    num = _seq_starts(seq_starts, x.shape[0], dev)
    dx, ddt, dB, dC = (torch.empty_like(t) if d is None else d for d, t in ((dx, x), (ddt, dt), (dB, B), (dC, C)))
    shape, code, layout, grads, nbytes, states = _scan_backward_plan(
        *metas, _meta(dO, "dO", dev), _meta(dx, "dx", dev), _meta(ddt, "ddt", dev, False), _meta(dB, "dB", dev),
        _meta(dC, "dC", dev), num)
    dA = torch.empty_like(A) if dA is None else dA
    dD = torch.empty_like(D) if dD is None and D is not None else dD
    ddt_bias = torch.empty_like(dt_bias) if ddt_bias is None and dt_bias is not None else ddt_bias
    for t, name in ((dA, "dA"), (dD, "dD"), (ddt_bias, "ddt_bias")):
        _norm_vector(t, name, H, torch.float32, dev)
    if S_init is not None and dS_init is None:
        dS_init = torch.empty_like(S_init)
    for t, name in ((S_init, "S_init"), (dS_final, "dS_final"), (dS_init, "dS_init")):
        if t is not None:
            _need(t, name, states, torch.float32, dev)
    ws = _workspace(nbytes, dev, workspace)
    opts = ScanOptions(_at(D), _at(dt_bias), bool(softplus), _at(S_init), _at(seq_starts), max(num, 0),
                       ctypes.pointer(layout))
    _launch(dev, "ttt_selective_scan_backward", lib().ttt_selective_scan_backward, shape, code, _at(x), _at(dt), _at(A),
            _at(B), _at(C), _at(dO), _at(dS_final), ctypes.byref(opts), ctypes.byref(grads), _at(dx), _at(ddt), _at(dA),
            _at(dB), _at(dC), _at(dD), _at(ddt_bias), _at(dS_init), _at(ws), nbytes)
    return dx, ddt, dA, dB, dC, dD, ddt_bias, dS_init


@functools.lru_cache(maxsize=256)
def _scan_step_shape(*sizes):
    return ctypes.byref(ScanStepShape(*sizes))


def ttt_selective_scan_step(x, dt, A, B, C, S, D=None, dt_bias=None, softplus=False, slots=None, O=None):
    """One token of the selective scan for each row of a serving batch.  x [rows, H, P], B, C [rows, G, N] of one dtype,
    dt [rows, H], A, D, dt_bias [H] fp32; S [states, H, P, N] fp32 is the pool of states, updated in place; slots
    [rows] int32 on the device names each row's state (a slot outside the pool, such as -1: a padding row, whose output
    is zero; rows of one slot go in row order; at most 65536 rows; None: row r's state is S[r]).  Returns O [rows, H,
    P]."""
    (R, H, P), (_, G, N), pool = x.shape, B.shape, S.shape[0]
    t, dev = x.dtype, x.device
    _need(x, "x", (R, H, P), t, dev)
    _need(dt, "dt", (R, H), torch.float32, dev)
    _scan_heads(A, D, dt_bias, H, dev)
    _need(B, "B", (R, G, N), t, dev)
    _need(C, "C", (R, G, N), t, dev)
    _need(S, "S", (pool, H, P, N), torch.float32, dev)
    if slots is not None:
        _need(slots, "slots", (R,), torch.int32, dev)
    if O is None:
        O = torch.empty_like(x)
    else:
        _need(O, "O", (R, H, P), t, dev)
    _launch(dev, "ttt_selective_scan_step", lib().ttt_selective_scan_step, _scan_step_shape(R, pool, H, G, P, N), _dt(t),
            _at(x), _at(dt), _at(A), _at(B), _at(C), _at(D), _at(dt_bias), bool(softplus), _at(S), _at(slots), _at(O))
    return O
