"""Python binding of libvdn (ctypes; argument marshalling only).

Every function has the name of its C entry point in include/vdn.h, takes
torch CUDA tensors (or None where the C call accepts NULL), passes their
device pointers and the current torch stream, and raises VdnError on any
status other than VDN_OK. All arithmetic happens in the library's kernels;
there is no fallback: if libvdn.so is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvdn.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "vdn.h")

VDN_OK, VDN_ERR_INVALID, VDN_ERR_UNSUPPORTED, VDN_ERR_CUDA, VDN_ERR_NUMERIC = range(5)
VDN_F32, VDN_BF16 = 0, 1
VDN_INFO_TIMEOUT = -1
_DTYPES = {"f32": VDN_F32, "bf16": VDN_BF16, VDN_F32: VDN_F32, VDN_BF16: VDN_BF16}
TORCH_DTYPE = {VDN_F32: torch.float32, VDN_BF16: torch.bfloat16}


class VdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class vdn_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "H", "T", "U", "dk", "dv", "n_text", "chunk", "anchors", "in_dtype", "out_dtype",
                 "beta_per_token", "decay_bridge")]

    @property
    def C(self) -> int:
        return -(-self.T // self.chunk) if self.T > 0 else 0


def make_shape(B, H, T, U, d, n_text, chunk=5, anchors=0, in_dtype="bf16", out_dtype=None,
               beta_per_token=False, decay_bridge=False) -> vdn_shape:
    in_dt = _DTYPES[in_dtype]
    out_dt = in_dt if out_dtype is None else _DTYPES[out_dtype]
    return vdn_shape(B, H, T, U, d, d, n_text, chunk, anchors, in_dt, out_dt, int(bool(beta_per_token)),
                     int(bool(decay_bridge)))


def shape_for(w, B=None, H=None) -> vdn_shape:
    """Shape of a synth.Workload (optionally with other batch/head counts)."""
    return make_shape(w.B if B is None else B, w.H if H is None else H, w.T, w.U, w.d, w.n_text,
                      w.chunk, w.anchors, w.dtype, beta_per_token=w.beta_per_token,
                      decay_bridge=getattr(w, "decay_bridge", False))


class vdn_out_gate(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p), ("eps", ctypes.c_float)]


def out_gate(gate, norm_weight, eps=1e-6):
    """The readout epilogue's arguments: gate logits [B,H,T,U,dv] (input dtype),
    RMSNorm weights [H,dv] float32, eps. Returns a vdn_out_gate (keep the
    tensors alive while it is in use)."""
    return vdn_out_gate(_ptr(gate), _ptr(norm_weight), float(eps))


def _og(og):
    return None if og is None else ctypes.cast(ctypes.pointer(og), _P)


_lib = None

_P = ctypes.c_void_p
_SIGS = {
    "vdn_frame_grams": [_P, _P, _P, _P, _P, _P, _P, _P],
    "vdn_frame_factor": [_P, _P, _P, _P, _P, _P, _P, _P],
    "vdn_chunk_compose": [_P, _P, _P, _P, _P, _P, _P, _P],
    "vdn_scan_fwd": [_P, _P, _P, _P, _P, _P],
    "vdn_scan_bwd": [_P, _P, _P, _P, _P, _P],
    "vdn_scan_bidir": [_P, _P, _P, _P, _P, _P, _P, _P, _P],
    "vdn_chunk_readout": [_P, _P, _P, _P, _P, _P, _P],
    "vdn_text_state": [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P],
    "vdn_forward": [_P] * 13 + [ctypes.c_size_t, _P, _P, _P, _P],
    "vdn_frame_invert": [_P, _P, _P, _P, _P],
    "vdn_text_state_noalloc": [_P, _P, _P, _P, _P, _P, _P],
    "vdn_forward_pipelined": [_P] * 13 + [ctypes.c_size_t, _P, ctypes.c_int32, _P, _P, _P, _P],
    "vdn_chunk_readout_gated": [_P] * 8,
    "vdn_chunk_readout_bridged": [_P] * 9,
    "vdn_selftest_wait": [_P, _P],
    "vdn_stream_segment": [_P] * 6 + [ctypes.c_longlong] + [_P] * 5 + [ctypes.c_size_t, _P, _P],
    "vdn_stream_segment_bridged": [_P] * 6 + [ctypes.c_longlong] + [_P] * 7 + [ctypes.c_size_t, _P, _P],
    "vdn_rotary": [_P, _P, _P, ctypes.c_int32, _P],
    "vdn_decay_attn_workspace_bytes": [_P],
    "vdn_decay_attn": [_P] * 10 + [ctypes.c_size_t, _P, _P],
    "vdn_decay_attn_backward_workspace_bytes": [_P],
    "vdn_decay_attn_backward": [_P] * 14 + [ctypes.c_size_t, _P, _P],
    "vdn_decay_step": [_P] * 10,
}


def lib() -> ctypes.CDLL:
    """Load libvdn.so (built in-tree by frame_wise_delta_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise VdnError(VDN_ERR_CUDA, f"{LIB_PATH} is missing; build it with "
                                         "`python -m frame_wise_delta_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        for name in ("vdn_text_state_workspace_bytes", "vdn_forward_workspace_bytes",
                     "vdn_stream_workspace_bytes", "vdn_decay_attn_workspace_bytes",
                     "vdn_decay_attn_backward_workspace_bytes"):
            fn = getattr(L, name)
            fn.argtypes = [_P]
            fn.restype = ctypes.c_size_t
        L.vdn_status_string.argtypes = [ctypes.c_int]
        L.vdn_status_string.restype = ctypes.c_char_p
        L.vdn_last_error.argtypes = []
        L.vdn_last_error.restype = ctypes.c_char_p
        L.vdn_version.argtypes = []
        L.vdn_version.restype = ctypes.c_int32
        _lib = L
    return _lib


def declared_symbols() -> list[str]:
    """Every function name that include/vdn.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(vdn_\w+)\s*\(", text)))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise VdnError(VDN_ERR_INVALID, "tensor is not on a CUDA device")
    if not t.is_contiguous():
        raise VdnError(VDN_ERR_INVALID, "tensor is not contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int):
    if status != VDN_OK:
        L = lib()
        name = L.vdn_status_string(status).decode()
        msg = L.vdn_last_error().decode()
        raise VdnError(status, f"{name}: {msg}")


def _shp(s: vdn_shape):
    return ctypes.cast(ctypes.pointer(s), _P)


def vdn_frame_grams(s, K, V, beta, A, Bm, info=None, stream=None):
    _check(lib().vdn_frame_grams(_shp(s), _ptr(K), _ptr(V), _ptr(beta), _ptr(A), _ptr(Bm), _ptr(info),
                                 _stream(stream)))


def vdn_frame_factor(s, A, Bm, alpha, M, J, info, stream=None):
    _check(lib().vdn_frame_factor(_shp(s), _ptr(A), _ptr(Bm), _ptr(alpha), _ptr(M), _ptr(J), _ptr(info),
                                  _stream(stream)))


def vdn_frame_invert(s, A, W, info, stream=None):
    _check(lib().vdn_frame_invert(_shp(s), _ptr(A), _ptr(W), _ptr(info), _stream(stream)))


def vdn_chunk_compose(s, M, J, Mf, Jf, Mb, Jb, stream=None):
    _check(lib().vdn_chunk_compose(_shp(s), _ptr(M), _ptr(J), _ptr(Mf), _ptr(Jf), _ptr(Mb), _ptr(Jb),
                                   _stream(stream)))


def vdn_scan_fwd(s, Mf, Jf, S_T, F, stream=None):
    _check(lib().vdn_scan_fwd(_shp(s), _ptr(Mf), _ptr(Jf), _ptr(S_T), _ptr(F), _stream(stream)))


def vdn_scan_bwd(s, Mb, Jb, S_T, G, stream=None):
    _check(lib().vdn_scan_bwd(_shp(s), _ptr(Mb), _ptr(Jb), _ptr(S_T), _ptr(G), _stream(stream)))


def vdn_scan_bidir(s, Mf, Jf, Mb, Jb, S_T, F, G, stream=None):
    _check(lib().vdn_scan_bidir(_shp(s), _ptr(Mf), _ptr(Jf), _ptr(Mb), _ptr(Jb), _ptr(S_T), _ptr(F),
                                _ptr(G), _stream(stream)))


def vdn_chunk_readout(s, Q, F, G, O, info=None, stream=None):
    _check(lib().vdn_chunk_readout(_shp(s), _ptr(Q), _ptr(F), _ptr(G), _ptr(O), _ptr(info),
                                   _stream(stream)))


def vdn_text_state_workspace_bytes(s) -> int:
    return int(lib().vdn_text_state_workspace_bytes(_shp(s)))


def vdn_text_state(s, Kx, Vx, beta_x, S_T, workspace, info, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().vdn_text_state(_shp(s), _ptr(Kx), _ptr(Vx), _ptr(beta_x), _ptr(S_T), _ptr(workspace),
                                nbytes, _ptr(info), _stream(stream)))


def vdn_text_state_noalloc(s, Kx, Vx, beta_x, S_T, info, stream=None):
    """vdn_text_state with the library's fixed device scratch instead of a workspace."""
    _check(lib().vdn_text_state_noalloc(_shp(s), _ptr(Kx), _ptr(Vx), _ptr(beta_x), _ptr(S_T), _ptr(info),
                                        _stream(stream)))


def vdn_forward_workspace_bytes(s) -> int:
    return int(lib().vdn_forward_workspace_bytes(_shp(s)))


def vdn_forward(s, Q, K, V, beta, alpha, Kx, Vx, beta_x, O, F, G, workspace, info, events=None,
                stream=None, og=None):
    """events: None or 7 torch.cuda.Event (enable_timing, already recorded once so
    that their CUDA handles exist) recorded by the library between the stages.
    og: None or an out_gate(...) for the gated RMSNorm readout epilogue."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ev = None
    if events is not None:
        handles = [e.cuda_event if e is not None else None for e in events]
        if any(e is not None and not h for e, h in zip(events, handles)):
            raise VdnError(VDN_ERR_INVALID, "stage events must have been recorded once (no CUDA handle yet)")
        arr = (ctypes.c_void_p * 7)(*handles)
        ev = ctypes.cast(arr, ctypes.c_void_p)
    _check(lib().vdn_forward(_shp(s), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(alpha), _ptr(Kx),
                             _ptr(Vx), _ptr(beta_x), _ptr(O), _ptr(F), _ptr(G), _ptr(workspace), nbytes,
                             _ptr(info), ev, _og(og), _stream(stream)))


def pipeline_events(groups: int):
    """The 8 + groups timing events vdn_forward_pipelined records (created
    here by torch and recorded once so that their CUDA handles exist)."""
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(8 + groups)]
    for e in evs:
        e.record()
    return evs


def vdn_forward_pipelined(s, Q, K, V, beta, alpha, Kx, Vx, beta_x, O, F, G, workspace, info, groups, aux,
                          events, stream=None, og=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    handles = [e.cuda_event for e in events]
    if len(handles) < 8 + groups or not all(handles):
        raise VdnError(VDN_ERR_INVALID, "need 8 + groups recorded events")
    arr = (ctypes.c_void_p * len(handles))(*handles)
    _check(lib().vdn_forward_pipelined(_shp(s), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(alpha), _ptr(Kx),
                                       _ptr(Vx), _ptr(beta_x), _ptr(O), _ptr(F), _ptr(G), _ptr(workspace),
                                       nbytes, _ptr(info), int(groups), _stream(aux),
                                       ctypes.cast(arr, ctypes.c_void_p), _og(og), _stream(stream)))


def vdn_chunk_readout_gated(s, Q, F, G, og, O, info=None, stream=None):
    _check(lib().vdn_chunk_readout_gated(_shp(s), _ptr(Q), _ptr(F), _ptr(G), _og(og), _ptr(O), _ptr(info),
                                         _stream(stream)))


def vdn_chunk_readout_bridged(s, Q, F, G, alpha, og, O, info=None, stream=None):
    """The chunk readout through the decay bridge (shape.decay_bridge = 1); og may be None."""
    _check(lib().vdn_chunk_readout_bridged(_shp(s), _ptr(Q), _ptr(F), _ptr(G), _ptr(alpha), _og(og), _ptr(O),
                                           _ptr(info), _stream(stream)))


def vdn_stream_workspace_bytes(s) -> int:
    return int(lib().vdn_stream_workspace_bytes(_shp(s)))


def vdn_stream_segment(s, Q, K, V, beta, alpha, frame0, S_prev, S_in, O, F, workspace, info, stream=None):
    """One segment of a live stream through the forward memory only (see vdn.h)."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().vdn_stream_segment(_shp(s), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(alpha), int(frame0),
                                    _ptr(S_prev), _ptr(S_in), _ptr(O), _ptr(F), _ptr(workspace), nbytes,
                                    _ptr(info), _stream(stream)))


def vdn_stream_segment_bridged(s, Q, K, V, beta, alpha, frame0, S_prev, S_in, alpha_prev, O, F, alpha_tail,
                               workspace, info, stream=None):
    """One stream segment read through the decay bridge (see vdn.h); alpha_prev
    None for the stream's first segment, alpha_tail None when not needed."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().vdn_stream_segment_bridged(_shp(s), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(alpha),
                                            int(frame0), _ptr(S_prev), _ptr(S_in), _ptr(alpha_prev), _ptr(O),
                                            _ptr(F), _ptr(alpha_tail), _ptr(workspace), nbytes, _ptr(info),
                                            _stream(stream)))


# ------------------------------------------------- token-level operators
class vdn_rotary_args(ctypes.Structure):
    _fields_ = [("grid_h", ctypes.c_int32), ("grid_w", ctypes.c_int32), ("dim_t", ctypes.c_int32),
                ("dim_h", ctypes.c_int32), ("dim_w", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("frame0", ctypes.c_int64), ("theta", ctypes.c_double),
                ("scale_t", ctypes.c_double), ("scale_h", ctypes.c_double), ("scale_w", ctypes.c_double),
                ("pos", ctypes.c_void_p)]


class vdn_rotary_io(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("x_stride", ctypes.c_int64 * 3),
                ("y_stride", ctypes.c_int64 * 3), ("rotate", ctypes.c_int32)]


_IO_WORDS = ctypes.c_int64 * 27  # three vdn_rotary_io: nine words each, `rotate` in the last one's low half


def _bad(text):
    raise VdnError(VDN_ERR_INVALID, text)


def _arg(t, dtype, shape, dev, name):
    """The pointer of a token-level operator's tensor (None for None, an int as
    it is): contiguous, of that type and shape, on the current device."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype != dtype or t.shape != shape:
        _bad(f"{name} is {t.dtype} {tuple(t.shape)}, not {dtype} {shape}")
    if t.get_device() != dev or not t.is_contiguous():
        _bad(f"{name} is not a contiguous tensor on the current CUDA device")
    return t.data_ptr()


def _raw(t, dev, name):
    """As _arg, for a buffer of any type and shape: (pointer, bytes)."""
    if t is None or isinstance(t, int):
        return t, 0
    if t.get_device() != dev or not t.is_contiguous():
        _bad(f"{name} is not a contiguous tensor on the current CUDA device")
    return t.data_ptr(), t.numel() * t.element_size()


def _word(t, dev):
    """The pointer of info: one int32 on the current device (None for None, an int as it is)."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype != torch.int32 or t.numel() < 1 or t.get_device() != dev:
        _bad(f"info is {t.dtype} {tuple(t.shape)}, not an int32 word on the current CUDA device")
    return t.data_ptr()


def _device():
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else torch.cuda.current_device()


def _on(stream, dev):
    """The stream's handle; the current stream of the current device for None."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def rotary(dim_t, dim_h, dim_w, grid=(0, 0), interleaved=True, inverse=False, frame0=0, theta=10000.0,
           scale=(1.0, 1.0, 1.0), pos=None):
    """The arguments of vdn_rotary: channels of each axis, the frame's token
    grid (rows, columns), or pos [B, T*U, 3] int32 with the position of every
    token (keep the tensor alive while the result is in use)."""
    if pos is not None and pos.dtype != torch.int32:
        raise VdnError(VDN_ERR_INVALID, f"pos is {pos.dtype}, not torch.int32")
    r = vdn_rotary_args(grid[0], grid[1], dim_t, dim_h, dim_w, int(bool(interleaved)), int(bool(inverse)), int(frame0),
                        float(theta), float(scale[0]), float(scale[1]), float(scale[2]), _ptr(pos))
    r.pos_tensor = pos
    return r


def _rows(t, shape, dtype, dev, name):
    """(pointer, batch, head and token strides) of a [B, H, T, U, d] tensor."""
    if t.shape != shape or t.dtype != dtype:
        _bad(f"{name} is {t.dtype} {tuple(t.shape)}, not {dtype} {shape}")
    sb, sh, st, su, sd = t.stride()
    if sd != 1:
        _bad(f"{name}'s channels are not contiguous")
    if shape[3] == 1:
        su = st
    elif shape[2] > 1 and st != su * shape[3] and t.numel():
        _bad(f"{name}'s frames do not follow each other")
    if t.get_device() != dev:
        _bad(f"{name} is not on the current CUDA device")
    return t.data_ptr(), sb, sh, su


def vdn_rotary(s, r, X, Y, rotate=None, stream=None):
    """Rotates the tensors X into Y (lists of up to three [B, H, T, U, d]
    tensors, token-major views included); rotate[i] = 0 copies X[i]."""
    n = len(X)
    if n != len(Y) or n > 3 or (rotate is not None and len(rotate) != n):
        _bad("X, Y and rotate: up to three tensors each, as many")
    dev = _device()
    shape, dtype = (s.B, s.H, s.T, s.U, s.dk), TORCH_DTYPE[s.in_dtype]
    pos = getattr(r, "pos_tensor", None)
    if pos is not None:
        _arg(pos, torch.int32, (s.B, s.T * s.U, 3), dev, "pos")
    words = []
    for i in range(n):
        x, xb, xh, xt = _rows(X[i], shape, dtype, dev, "X")
        y, yb, yh, yt = _rows(Y[i], shape, dtype, dev, "Y")
        words += (x, y, xb, xh, xt, yb, yh, yt, 1 if rotate is None else rotate[i] & 0xFFFFFFFF)
    io = _IO_WORDS(*words)
    _check(lib().vdn_rotary(ctypes.byref(s), ctypes.byref(r), ctypes.byref(io), n, _on(stream, dev)))


def vdn_decay_attn_workspace_bytes(s) -> int:
    return int(lib().vdn_decay_attn_workspace_bytes(_shp(s)))


def vdn_decay_attn_backward_workspace_bytes(s) -> int:
    return int(lib().vdn_decay_attn_backward_workspace_bytes(_shp(s)))


def vdn_decay_attn(s, Q, K, V, log_decay, lens, S_in, O, S_out, workspace, info=None, stream=None):
    """Linear attention with one decay per head over the T * U tokens (see vdn.h); lens, S_in, S_out may be None."""
    dev = _device()
    x, st = (s.B, s.H, s.T, s.U, s.dk), (s.B, s.H, s.dv, s.dk)
    ti, to, f = TORCH_DTYPE[s.in_dtype], TORCH_DTYPE[s.out_dtype], torch.float32
    ws, n = _raw(workspace, dev, "workspace")
    _check(lib().vdn_decay_attn(
        ctypes.byref(s), _arg(Q, ti, x, dev, "Q"), _arg(K, ti, x, dev, "K"), _arg(V, ti, x, dev, "V"),
        _arg(log_decay, f, (s.H,), dev, "log_decay"), _arg(lens, torch.int32, (s.B,), dev, "lens"),
        _arg(S_in, f, st, dev, "S_in"), _arg(O, to, x, dev, "O"), _arg(S_out, f, st, dev, "S_out"), ws, n,
        _word(info, dev), _on(stream, dev)))


def vdn_decay_attn_backward(s, Q, K, V, log_decay, lens, S_in, dO, dS_out, dQ, dK, dV, dS_in, workspace, info=None,
                            stream=None):
    """Gradients of vdn_decay_attn (see vdn.h); lens, S_in, dS_out, dS_in may be None."""
    dev = _device()
    x, st = (s.B, s.H, s.T, s.U, s.dk), (s.B, s.H, s.dv, s.dk)
    ti, f = TORCH_DTYPE[s.in_dtype], torch.float32
    ws, n = _raw(workspace, dev, "workspace")
    _check(lib().vdn_decay_attn_backward(
        ctypes.byref(s), _arg(Q, ti, x, dev, "Q"), _arg(K, ti, x, dev, "K"), _arg(V, ti, x, dev, "V"),
        _arg(log_decay, f, (s.H,), dev, "log_decay"), _arg(lens, torch.int32, (s.B,), dev, "lens"),
        _arg(S_in, f, st, dev, "S_in"), _arg(dO, ti, x, dev, "dO"), _arg(dS_out, f, st, dev, "dS_out"),
        _arg(dQ, ti, x, dev, "dQ"), _arg(dK, ti, x, dev, "dK"), _arg(dV, ti, x, dev, "dV"), _arg(dS_in, f, st, dev, "dS_in"),
        ws, n, _word(info, dev), _on(stream, dev)))


def vdn_decay_step(s, Q, K, V, log_decay, active, S_in, O, S_out, stream=None):
    """One token per sequence of vdn_decay_attn (see vdn.h); Q, K, V, O [B, H, d], S_out may be S_in."""
    dev = _device()
    x, st = (s.B, s.H, s.dk), (s.B, s.H, s.dv, s.dk)
    ti, to, f = TORCH_DTYPE[s.in_dtype], TORCH_DTYPE[s.out_dtype], torch.float32
    _check(lib().vdn_decay_step(
        ctypes.byref(s), _arg(Q, ti, x, dev, "Q"), _arg(K, ti, x, dev, "K"), _arg(V, ti, x, dev, "V"),
        _arg(log_decay, f, (s.H,), dev, "log_decay"), _arg(active, torch.int32, (s.B,), dev, "active"),
        _arg(S_in, f, st, dev, "S_in"), _arg(O, to, x, dev, "O"), _arg(S_out, f, st, dev, "S_out"), _on(stream, dev)))


def vdn_selftest_wait(info, stream=None):
    """Self-test of the bounded pipeline waits (see vdn.h): *info becomes VDN_INFO_TIMEOUT."""
    _check(lib().vdn_selftest_wait(_ptr(info), _stream(stream)))


def vdn_status_string(status: int) -> str:
    return lib().vdn_status_string(status).decode()


def vdn_last_error() -> str:
    return lib().vdn_last_error().decode()


def vdn_version() -> int:
    return int(lib().vdn_version())


# ------------------------------------------------------------------ helpers
def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte-aligned uint8 device buffer of at least nbytes bytes."""
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)


class Stream:
    """A live stream read through the forward memory: call with each segment's
    frames (whole chunks except the last); the carried states (the forward
    states before the last two chunks) start as the text state S^T."""

    def __init__(self, s: vdn_shape, S_T: torch.Tensor, device="cuda"):
        self.s = s
        self.ws = workspace(vdn_stream_workspace_bytes(s), device)
        self.info = torch.zeros(1, dtype=torch.int32, device=device)
        self.O = torch.empty((s.B, s.H, s.T, s.U, s.dv), dtype=TORCH_DTYPE[s.out_dtype], device=device)
        self.F = torch.empty((s.B, s.H, s.C + 1, s.dv, s.dk), dtype=torch.float32, device=device)
        self.S_prev = S_T.clone()
        self.S_in = S_T.clone()
        self.frame0 = 0
        # with the decay bridge: the last chunk's decay product, carried too
        self.alpha_tail = (torch.ones((s.B, s.H, s.dk), dtype=torch.float32, device=device)
                           if s.decay_bridge else None)

    def __call__(self, Q, K, V, beta, alpha, stream=None):
        if self.s.decay_bridge:
            prev = None if self.frame0 == 0 else self.alpha_tail.clone()
            vdn_stream_segment_bridged(self.s, Q, K, V, beta, alpha, self.frame0, self.S_prev, self.S_in, prev,
                                       self.O, self.F, self.alpha_tail, self.ws, self.info, stream)
        else:
            vdn_stream_segment(self.s, Q, K, V, beta, alpha, self.frame0, self.S_prev, self.S_in, self.O,
                               self.F, self.ws, self.info, stream)
        C = self.s.C
        if C > 0:
            self.S_prev.copy_(self.F[:, :, C - 1])
            self.S_in.copy_(self.F[:, :, C])
        self.frame0 += self.s.T
        return self.O


class Forward:
    """Preallocated buffers for repeated vdn_forward calls on one shape."""

    def __init__(self, s: vdn_shape, device="cuda", keep_states=True):
        self.s = s
        BH = s.B * s.H
        C = s.C
        self.ws = workspace(vdn_forward_workspace_bytes(s), device)
        self.info = torch.zeros(1, dtype=torch.int32, device=device)
        out_dt = TORCH_DTYPE[s.out_dtype]
        self.O = torch.empty((s.B, s.H, s.T, s.U, s.dv), dtype=out_dt, device=device)
        self.F = self.G = None
        if keep_states:
            self.F = torch.empty((s.B, s.H, C + 1, s.dv, s.dk), dtype=torch.float32, device=device)
            self.G = torch.empty_like(self.F)
        del BH

    def __call__(self, Q, K, V, beta, alpha, Kx, Vx, beta_x, events=None, stream=None, og=None):
        vdn_forward(self.s, Q, K, V, beta, alpha, Kx, Vx, beta_x, self.O, self.F, self.G, self.ws,
                    self.info, events, stream, og)
        return self.O


class PipelinedForward(Forward):
    """vdn_forward_pipelined with its own auxiliary stream and events."""

    def __init__(self, s: vdn_shape, groups: int = 3, device="cuda", keep_states=True):
        super().__init__(s, device, keep_states)
        self.groups = groups
        self.aux = torch.cuda.Stream(device=device)
        self.events = pipeline_events(groups)

    def __call__(self, Q, K, V, beta, alpha, Kx, Vx, beta_x, events=None, stream=None, og=None):
        vdn_forward_pipelined(self.s, Q, K, V, beta, alpha, Kx, Vx, beta_x, self.O, self.F, self.G, self.ws,
                              self.info, self.groups, self.aux, self.events, stream, og)
        return self.O
