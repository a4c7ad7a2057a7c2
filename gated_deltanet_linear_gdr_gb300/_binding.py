"""Thin ctypes binding over libgdr.so (include/gdr.h).

Argument marshalling only: tensors are checked for dtype/device/shape, their
data pointers and strides are packed into gdr_step_args, and the C entry point
of the same name runs every step of the path on the GPU.  PyTorch supplies the
device memory and the current stream; nothing here computes.

If libgdr.so is missing the first call raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdr.so")

GDR_OK, GDR_ERR_INVALID_ARG, GDR_ERR_UNSUPPORTED, GDR_ERR_CUDA = 0, -1, -2, -3
GDR_F32, GDR_BF16 = 0, 1
STATUS_BITS = {
    0x1: "BAD_SLOT", 0x2: "BAD_OFFSETS", 0x4: "BAD_RING_SLOT", 0x8: "BAD_COUNT",
    0x10: "ROW_TOO_LONG", 0x20: "BAD_ACCEPTED", 0x40: "SNAPSHOT_OVERFLOW", 0x80: "BAD_DECAY",
    0x100: "TIMEOUT", 0x200: "NO_MASS",
}


class GdrError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"gdr error {code}: {msg}")
        self.code = code


class gdr_host_io(ctypes.Structure):
    """Mirror of struct gdr_host_io in include/gdr.h (host pointers)."""
    _fields_ = [
        ("qkv", ctypes.c_void_p), ("decay", ctypes.c_void_p), ("beta", ctypes.c_void_p),
        ("slot_idx", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("out", ctypes.c_void_p),
    ]


class gdr_step_args(ctypes.Structure):
    """Mirror of struct gdr_step_args in include/gdr.h (same order and types)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("nv", ctypes.c_int32), ("nk", ctypes.c_int32),
        ("K", ctypes.c_int32), ("V", ctypes.c_int32),
        ("decay_is_log", ctypes.c_int32), ("use_qk_l2norm", ctypes.c_int32),
        ("state_dtype", ctypes.c_int32),
        ("total_tokens", ctypes.c_int64), ("max_row_len", ctypes.c_int64),
        ("qkv", ctypes.c_void_p), ("qkv_seq_stride", ctypes.c_int64),
        ("qkv_chan_stride", ctypes.c_int64),
        ("decay", ctypes.c_void_p), ("beta", ctypes.c_void_p),
        ("tok_seq_stride", ctypes.c_int64), ("tok_head_stride", ctypes.c_int64),
        ("scale", ctypes.c_float), ("eps", ctypes.c_float),
        ("out", ctypes.c_void_p), ("out_seq_stride", ctypes.c_int64),
        ("out_vdim_stride", ctypes.c_int64),
        ("state", ctypes.c_void_p), ("state_slot_stride", ctypes.c_int64),
        ("state_head_stride", ctypes.c_int64), ("state_kdim_stride", ctypes.c_int64),
        ("state_vdim_stride", ctypes.c_int64), ("max_slots", ctypes.c_int64),
        ("slot_idx", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
        ("beta_seq_stride", ctypes.c_int64), ("beta_head_stride", ctypes.c_int64),
        ("beta_vdim_stride", ctypes.c_int64),
    ]


class gdr_conv_args(ctypes.Structure):
    """Mirror of struct gdr_conv_args in include/gdr.h."""
    _fields_ = [
        ("width", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("weight", ctypes.c_void_p), ("weight_chan_stride", ctypes.c_int64),
        ("weight_tap_stride", ctypes.c_int64), ("bias", ctypes.c_void_p),
        ("conv_state", ctypes.c_void_p), ("state_slot_stride", ctypes.c_int64),
        ("state_chan_stride", ctypes.c_int64), ("state_tap_stride", ctypes.c_int64),
    ]


class gdr_linattn_args(ctypes.Structure):
    """Mirror of struct gdr_linattn_args in include/gdr.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("nv", ctypes.c_int32), ("nk", ctypes.c_int32), ("K", ctypes.c_int32),
        ("V", ctypes.c_int32), ("decay_is_log", ctypes.c_int32), ("token_dtype", ctypes.c_int32),
        ("state_dtype", ctypes.c_int32), ("total_tokens", ctypes.c_int64), ("max_row_len", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("q_seq_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("k", ctypes.c_void_p), ("k_seq_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
        ("v", ctypes.c_void_p), ("v_seq_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
        ("decay", ctypes.c_void_p), ("decay_stride", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_seq_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("state", ctypes.c_void_p), ("state_slot_stride", ctypes.c_int64), ("state_head_stride", ctypes.c_int64),
        ("state_kdim_stride", ctypes.c_int64), ("state_vdim_stride", ctypes.c_int64), ("max_slots", ctypes.c_int64),
        ("slot_idx", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64), ("scale", ctypes.c_float),
    ]


class gdr_norm_args(ctypes.Structure):
    """Mirror of struct gdr_norm_args in include/gdr.h."""
    _fields_ = [
        ("tokens", ctypes.c_int64), ("heads", ctypes.c_int32), ("D", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("gate_first", ctypes.c_int32),
        ("has_post_norm", ctypes.c_int32), ("has_pre_norm", ctypes.c_int32), ("centered", ctypes.c_int32),
        ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
        ("x", ctypes.c_void_p), ("x_seq_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
        ("gate", ctypes.c_void_p), ("gate_seq_stride", ctypes.c_int64), ("gate_head_stride", ctypes.c_int64),
        ("gate_elem_stride", ctypes.c_int64),
        ("residual", ctypes.c_void_p), ("residual_seq_stride", ctypes.c_int64),
        ("residual_head_stride", ctypes.c_int64),
        ("residual_out", ctypes.c_void_p), ("residual_out_seq_stride", ctypes.c_int64),
        ("residual_out_head_stride", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_seq_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("post_weight", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
    ]


class gdr_short_conv_args(ctypes.Structure):
    """Mirror of struct gdr_short_conv_args in include/gdr.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("channels", ctypes.c_int32), ("width", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("token_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("keep_state", ctypes.c_int32),
        ("total_tokens", ctypes.c_int64), ("max_row_len", ctypes.c_int64),
        ("x", ctypes.c_void_p), ("x_seq_stride", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("weight_chan_stride", ctypes.c_int64), ("weight_tap_stride", ctypes.c_int64),
        ("bias", ctypes.c_void_p), ("out", ctypes.c_void_p), ("out_seq_stride", ctypes.c_int64),
        ("conv_state", ctypes.c_void_p), ("state_slot_stride", ctypes.c_int64), ("state_chan_stride", ctypes.c_int64),
        ("state_tap_stride", ctypes.c_int64), ("max_slots", ctypes.c_int64),
        ("slot_idx", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("counts", ctypes.c_void_p),
    ]


class gdr_scan_args(ctypes.Structure):
    """Mirror of struct gdr_scan_args in include/gdr.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("nv", ctypes.c_int32), ("nk", ctypes.c_int32), ("K", ctypes.c_int32),
        ("V", ctypes.c_int32), ("dt_softplus", ctypes.c_int32), ("token_dtype", ctypes.c_int32),
        ("dt_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("keep_state", ctypes.c_int32),
        ("total_tokens", ctypes.c_int64), ("max_row_len", ctypes.c_int64),
        ("x", ctypes.c_void_p), ("x_seq_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
        ("dt", ctypes.c_void_p), ("dt_seq_stride", ctypes.c_int64), ("dt_head_stride", ctypes.c_int64),
        ("dt_elem_stride", ctypes.c_int64),
        ("B", ctypes.c_void_p), ("B_seq_stride", ctypes.c_int64), ("B_head_stride", ctypes.c_int64),
        ("C", ctypes.c_void_p), ("C_seq_stride", ctypes.c_int64), ("C_head_stride", ctypes.c_int64),
        ("z", ctypes.c_void_p), ("z_seq_stride", ctypes.c_int64), ("z_head_stride", ctypes.c_int64),
        ("A", ctypes.c_void_p), ("A_head_stride", ctypes.c_int64), ("A_kdim_stride", ctypes.c_int64),
        ("A_vdim_stride", ctypes.c_int64),
        ("D", ctypes.c_void_p), ("D_head_stride", ctypes.c_int64), ("D_vdim_stride", ctypes.c_int64),
        ("dt_bias", ctypes.c_void_p), ("dt_bias_head_stride", ctypes.c_int64), ("dt_bias_vdim_stride", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_seq_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("state", ctypes.c_void_p), ("state_slot_stride", ctypes.c_int64), ("state_head_stride", ctypes.c_int64),
        ("state_kdim_stride", ctypes.c_int64), ("state_vdim_stride", ctypes.c_int64), ("max_slots", ctypes.c_int64),
        ("slot_idx", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("counts", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
    ]


class gdr_accept_args(ctypes.Structure):
    """Mirror of struct gdr_accept_args in include/gdr.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("vocab", ctypes.c_int32), ("prob_dtype", ctypes.c_int32), ("max_row_len", ctypes.c_int32),
        ("total_tokens", ctypes.c_int64),
        ("target", ctypes.c_void_p), ("target_seq_stride", ctypes.c_int64),
        ("draft", ctypes.c_void_p), ("draft_seq_stride", ctypes.c_int64),
        ("tokens", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("uniforms", ctypes.c_void_p),
        ("row_uniforms", ctypes.c_void_p), ("out_tokens", ctypes.c_void_p), ("out_seq_stride", ctypes.c_int64),
        ("counts", ctypes.c_void_p),
    ]


def _packer(cls):
    """Packs a call's values into the bytes of `cls` in one step (a ctypes
    structure costs several microseconds to fill; a decode step's call is
    bound by what the host does)."""
    codes = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_void_p: "P", ctypes.c_float: "f"}
    p = struct.Struct("@" + "".join(codes[t] for _, t in cls._fields_) + "0q")
    assert p.size == ctypes.sizeof(cls)
    return p.pack


_pack_linattn = _packer(gdr_linattn_args)
_pack_norm = _packer(gdr_norm_args)
_pack_short_conv = _packer(gdr_short_conv_args)
_pack_scan = _packer(gdr_scan_args)
_pack_accept = _packer(gdr_accept_args)

_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libgdr.so (built by gated_deltanet_linear_gdr_gb300.build)."""
    global _lib
    with _lock:
        if _lib is None or path is not None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(
                    f"{p} is missing: build it with `python -c \"import __graft_entry__ as g; "
                    f"g.build()\"` (the GDR path has no CPU or Python fallback)")
            lib = ctypes.CDLL(p)
            A = ctypes.POINTER(gdr_step_args)
            vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            sig = {
                "gdr_last_error": ([], ctypes.c_char_p),
                "gdr_version": ([], ctypes.c_int),
                "gdr_output_shape": ([i64, i32, i32, ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
                "gdr_ring_record_elements": ([i32, i32, i32], ctypes.c_int),
                "gdr_fwd": ([A, vp], ctypes.c_int),
                "gdr_fwd_host": ([A, ctypes.POINTER(gdr_host_io), i32, vp, vp, vp], ctypes.c_int),
                "gdr_fwd_host_noalloc": ([A, ctypes.POINTER(gdr_host_io), i32, vp, vp, vp], ctypes.c_int),
                "gdr_fwd_dense": ([A, vp, vp, vp], ctypes.c_int),
                "gdr_fwd_conv": ([A, ctypes.POINTER(gdr_conv_args), vp], ctypes.c_int),
                "gdr_verify_ring": ([A, vp, i32, i64, i32, i64, vp, vp], ctypes.c_int),
                "gdr_fold": ([A, vp, i32, i64, i32, i64, vp, vp, vp], ctypes.c_int),
                "gdr_fwd_snapshots": ([A, vp, i64, i64, i64, i32, i32, vp], ctypes.c_int),
                "gdr_rollback": ([A, vp, i64, i64, i64, i32, vp, vp], ctypes.c_int),
                "gdr_linattn_fwd": ([vp, vp], ctypes.c_int),  # structs as packed bytes or by reference
                "gdr_linattn_workspace_bytes": ([vp], ctypes.c_int64),
                "gdr_block_norm": ([vp, vp], ctypes.c_int),
                "gdr_short_conv": ([vp, vp], ctypes.c_int),
                "gdr_selective_scan": ([vp, vp], ctypes.c_int),
                "gdr_selective_scan_workspace_bytes": ([vp], ctypes.c_int64),
                "gdr_accept_drafts": ([vp, vp], ctypes.c_int),
                "gdr_get_status": ([ctypes.POINTER(ctypes.c_uint32), i32], ctypes.c_int),
                "gdr_probe_fma": ([i32, i32, i32, vp, i64, ctypes.POINTER(ctypes.c_int32), vp], ctypes.c_int),
            }
            for name, (args, res) in sig.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            if path is None:
                _lib = lib
            else:
                return lib
    return _lib


def _check(rc: int):
    if rc != GDR_OK:
        msg = load_library().gdr_last_error().decode(errors="replace")
        raise GdrError(rc, msg)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t


def _ring_dtype(ring: torch.Tensor) -> int:
    return GDR_BF16 if ring.dtype == torch.bfloat16 else GDR_F32


def _state_dtype(state: torch.Tensor) -> int:
    if state.dtype == torch.bfloat16:
        return GDR_BF16
    if state.dtype == torch.float32:
        return GDR_F32
    raise TypeError(f"state dtype {state.dtype}: expected bfloat16 or float32")


def make_args(qkv, decay, beta, state, slot_idx, offsets, out, *, nk: int,
              decay_is_log=False, use_qk_l2norm=True, scale=0.0, eps=1e-6,
              max_row_len=0) -> gdr_step_args:
    """Pack tensors into gdr_step_args (no copies; strides passed through)."""
    _dev(state, "state", (torch.bfloat16, torch.float32))
    if state.dim() != 4:
        raise ValueError("state must be [max_slots, nv, K, V]")
    max_slots, nv, K, V = state.shape
    _dev(slot_idx, "slot_idx", torch.int32)
    batch = slot_idx.shape[0]
    a = gdr_step_args()
    a.batch, a.nv, a.nk, a.K, a.V = batch, nv, nk, K, V
    a.decay_is_log, a.use_qk_l2norm = int(bool(decay_is_log)), int(bool(use_qk_l2norm))
    a.state_dtype = _state_dtype(state)
    a.max_row_len = int(max_row_len)
    a.scale, a.eps = float(scale), float(eps)
    a.state = state.data_ptr()
    (a.state_slot_stride, a.state_head_stride, a.state_kdim_stride,
     a.state_vdim_stride) = state.stride()
    a.max_slots = max_slots
    a.slot_idx = slot_idx.data_ptr()
    if qkv is not None:
        _dev(qkv, "qkv", torch.float32)
        _dev(decay, "decay", torch.float32)
        _dev(beta, "beta", torch.float32)
        _dev(out, "out", torch.float32)
        _dev(offsets, "offsets", torch.int32)
        T = qkv.shape[0]
        if qkv.shape[1] != 2 * nk * K + nv * V:
            raise ValueError(f"qkv has {qkv.shape[1]} channels, expected 2*nk*K + nv*V = "
                             f"{2 * nk * K + nv * V}")
        if decay.shape != (T, nv):
            raise ValueError("decay must be [T, nv]")
        if beta.shape == (T, nv, V):
            # per value element ("core.ssm.ops.gdp.fused_recurrent", beta [B, T, HV, V])
            a.beta_seq_stride, a.beta_head_stride, a.beta_vdim_stride = beta.stride()
            if a.beta_vdim_stride <= 0:
                raise ValueError("per-element beta needs a positive value-dim stride")
        elif beta.shape != (T, nv) or decay.stride() != beta.stride():
            raise ValueError("beta must be [T, nv] with decay's strides, or [T, nv, V]")
        if out.shape != (T, nv * V):
            raise ValueError(f"out must be [T, nv*V] = [{T}, {nv * V}]")
        if offsets.shape != (batch + 1,) or not offsets.is_contiguous():
            raise ValueError("offsets must be a contiguous [batch+1] int32 tensor")
        a.total_tokens = T
        a.qkv = qkv.data_ptr()
        a.qkv_seq_stride, a.qkv_chan_stride = qkv.stride()
        a.decay, a.beta = decay.data_ptr(), beta.data_ptr()
        a.tok_seq_stride, a.tok_head_stride = decay.stride()
        a.out = out.data_ptr()
        a.out_seq_stride, a.out_vdim_stride = out.stride()
        a.offsets = offsets.data_ptr()
    if not slot_idx.is_contiguous():
        raise ValueError("slot_idx must be contiguous")
    return a


def _nk_from_qkv(qkv, state):
    nv, K, V = state.shape[1:]
    rest = qkv.shape[1] - nv * V
    if rest <= 0 or rest % (2 * K):
        raise ValueError("cannot infer nk from qkv channels")
    return rest // (2 * K)


def gdr_output_shape(total_tokens: int, nv: int, V: int):
    shp = (ctypes.c_int64 * 2)()
    _check(load_library().gdr_output_shape(total_tokens, nv, V, shp))
    return int(shp[0]), int(shp[1])


def gdr_ring_record_elements(K: int, V: int, ratio: int) -> int:
    n = load_library().gdr_ring_record_elements(K, V, ratio)
    if n < 0:
        _check(n)
    return n


def gdr_fwd(qkv, decay, beta, state, slot_idx, offsets, out=None, *, decay_is_log=False,
            use_qk_l2norm=True, scale=0.0, eps=1e-6, max_row_len=0):
    """Forward pass ("gated_delta_recurrence_fwd_gpu"); state updated in place; returns out."""
    if out is None:
        out = torch.empty(gdr_output_shape(qkv.shape[0], state.shape[1], state.shape[3]),
                          dtype=torch.float32, device=qkv.device)
    a = make_args(qkv, decay, beta, state, slot_idx, offsets, out, nk=_nk_from_qkv(qkv, state),
                  decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps,
                  max_row_len=max_row_len)
    _check(load_library().gdr_fwd(ctypes.byref(a), _stream(qkv.device)))
    return out


def _host(t: torch.Tensor, name: str, dtype):
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError(f"{name} must be a host (CPU) torch.Tensor")
    if t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor")
    return t


class HostForward:
    """gdr_fwd_host for host-resident tokens: the forward pass
    ("gated_delta_recurrence_fwd_gpu") with the tokens copied in and the
    output copied back inside one C-ABI call, row groups pipelined over three
    streams (copies in, compute, copies out).

    Owns the device staging buffers for batches of up to `batch` rows and
    `total_tokens` tokens and the two side streams; the pool stays the
    caller's device tensor.  Host tensors should be pinned
    (tensor.pin_memory()) for the copies to overlap the compute."""

    def __init__(self, state, nk: int, batch: int, total_tokens: int, *, decay_is_log=False,
                 use_qk_l2norm=True, scale=0.0, eps=1e-6, max_row_len=0, chunks=0):
        _dev(state, "state", (torch.bfloat16, torch.float32))
        dev = state.device
        nv, K, V = state.shape[1:]
        f32, i32 = torch.float32, torch.int32
        self.state = state
        self.qkv = torch.empty((total_tokens, 2 * nk * K + nv * V), dtype=f32, device=dev)
        self.decay = torch.empty((total_tokens, nv), dtype=f32, device=dev)
        self.beta = torch.empty((total_tokens, nv), dtype=f32, device=dev)
        self.out = torch.empty((total_tokens, nv * V), dtype=f32, device=dev)
        self.slot_idx = torch.empty((batch,), dtype=i32, device=dev)
        self.offsets = torch.empty((batch + 1,), dtype=i32, device=dev)
        self.h2d = torch.cuda.Stream(dev)
        self.d2h = torch.cuda.Stream(dev)
        self.chunks = int(chunks)
        self.args = make_args(self.qkv, self.decay, self.beta, state, self.slot_idx, self.offsets, self.out,
                              nk=nk, decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale,
                              eps=eps, max_row_len=max_row_len)
        self.device = dev

    def __call__(self, qkv, decay, beta, slot_idx, offsets, out, stream: Optional[int] = None):
        """Runs the pass on host tensors; `out` (host, [T, nv*V]) holds the
        result once `stream` (default: the current stream) has passed the call."""
        for t, n, d in ((qkv, "qkv", torch.float32), (decay, "decay", torch.float32),
                        (beta, "beta", torch.float32), (slot_idx, "slot_idx", torch.int32),
                        (offsets, "offsets", torch.int32), (out, "out", torch.float32)):
            _host(t, n, d)
        if tuple(qkv.shape) != tuple(self.qkv.shape) or tuple(out.shape) != tuple(self.out.shape):
            raise ValueError("qkv / out shapes differ from the staging buffers")
        if slot_idx.shape[0] != self.slot_idx.shape[0] or offsets.shape[0] != self.offsets.shape[0]:
            raise ValueError("slot_idx / offsets lengths differ from the staging buffers")
        io = gdr_host_io(qkv.data_ptr(), decay.data_ptr(), beta.data_ptr(), slot_idx.data_ptr(),
                         offsets.data_ptr(), out.data_ptr())
        s = _stream(self.device) if stream is None else stream
        _check(load_library().gdr_fwd_host(ctypes.byref(self.args), ctypes.byref(io), self.chunks, s,
                                           self.h2d.cuda_stream, self.d2h.cuda_stream))
        return out


def make_conv_args(weight, bias, conv_state, state, activation="silu") -> gdr_conv_args:
    """Pack the Pass-1 convolution's tensors into gdr_conv_args: weight
    [conv_dim, width] float32, bias [conv_dim] float32 or None, conv_state
    [slots, conv_dim, width-1] float32 indexed like the pool `state` (None
    when width == 1); activation "silu" or None."""
    _dev(weight, "conv_weight", torch.float32)
    if weight.dim() != 2:
        raise ValueError("conv_weight must be [conv_dim, width]")
    C, width = weight.shape
    c = gdr_conv_args()
    c.width = width
    if activation not in (None, "silu"):
        raise ValueError('activation must be "silu" or None')
    c.activation = 1 if activation == "silu" else 0
    c.weight = weight.data_ptr()
    c.weight_chan_stride, c.weight_tap_stride = weight.stride()
    if bias is not None:
        _dev(bias, "conv_bias", torch.float32)
        if bias.shape != (C,) or bias.stride() != (1,):
            raise ValueError("conv_bias must be a contiguous [conv_dim] tensor")
        c.bias = bias.data_ptr()
    if width > 1:
        if conv_state is None:
            raise ValueError("conv_state is needed for width > 1")
        _dev(conv_state, "conv_state", torch.float32)
        if conv_state.dim() != 3 or conv_state.shape[1:] != (C, width - 1):
            raise ValueError(f"conv_state must be [slots, {C}, {width - 1}]")
        if conv_state.shape[0] < state.shape[0]:
            raise ValueError("conv_state needs one row per pool slot (it is indexed by slot_idx)")
        c.conv_state = conv_state.data_ptr()
        c.state_slot_stride, c.state_chan_stride, c.state_tap_stride = conv_state.stride()
    return c


def gdr_fwd_conv(x, decay, beta, state, slot_idx, offsets, conv_weight, conv_bias=None, conv_state=None,
                 activation="silu", out=None, *, decay_is_log=False, use_qk_l2norm=True, scale=0.0, eps=1e-6,
                 max_row_len=0):
    """Forward pass on the raw Pass-1 input x [T, 2*nk*K + nv*V]: the causal
    depthwise convolution ("gated_delta_recurrence_fwd_gpu", Args:
    qkv_conv_output is the Conv1d output from Pass 1) fused into the
    recurrence's operand staging; state and conv_state updated in place;
    returns out."""
    if out is None:
        out = torch.empty(gdr_output_shape(x.shape[0], state.shape[1], state.shape[3]),
                          dtype=torch.float32, device=x.device)
    a = make_args(x, decay, beta, state, slot_idx, offsets, out, nk=_nk_from_qkv(x, state),
                  decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps,
                  max_row_len=max_row_len)
    if conv_weight.shape[0] != x.shape[1]:
        raise ValueError("conv_weight must have one row per input channel")
    c = make_conv_args(conv_weight, conv_bias, conv_state, state, activation)
    _check(load_library().gdr_fwd_conv(ctypes.byref(a), ctypes.byref(c), _stream(x.device)))
    return out


def prepare_fwd_conv(x, decay, beta, state, slot_idx, offsets, conv_weight, conv_bias, conv_state, out, *,
                     activation="silu", decay_is_log=False, use_qk_l2norm=True, scale=0.0, eps=1e-6,
                     max_row_len=0) -> "Prepared":
    a = make_args(x, decay, beta, state, slot_idx, offsets, out, nk=_nk_from_qkv(x, state),
                  decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps,
                  max_row_len=max_row_len)
    c = make_conv_args(conv_weight, conv_bias, conv_state, state, activation)
    lib = load_library()
    return Prepared(lambda ap, cp, s: lib.gdr_fwd_conv(ap, cp, s), a, (ctypes.byref(c),),
                    (x, decay, beta, state, slot_idx, offsets, out, conv_weight, conv_bias, conv_state, c),
                    x.device)


def gdr_fwd_dense(qkv, decay, beta, offsets, initial_state=None, output_final_state=True, out=None, *,
                  nv=None, K=None, state_dtype=torch.float32, decay_is_log=False, use_qk_l2norm=True,
                  scale=0.0, eps=1e-6, max_row_len=0):
    """Forward pass with a dense start / end state ("core.ssm.ops.gdp.fused_recurrent",
    initial_state [N, HV, K, V] or None for zeros, output_final_state).  Returns
    (out, final_state); final_state is a new [N, HV, K, V] tensor of the start
    state's dtype (None unless output_final_state).  Without an initial state,
    nv and K (= V) give the shape and state_dtype the dtype."""
    batch = offsets.shape[0] - 1
    if initial_state is not None:
        ref = initial_state
    else:
        if nv is None or K is None:
            raise ValueError("without initial_state, nv and K are needed")
        ref = torch.empty((batch, nv, K, K), dtype=state_dtype, device=qkv.device)
    final = torch.empty_like(ref, memory_format=torch.contiguous_format) if output_final_state else None
    if initial_state is not None and final is not None and final.stride() != initial_state.stride():
        raise ValueError("initial_state must be contiguous (final_state shares its strides)")
    if out is None:
        out = torch.empty(gdr_output_shape(qkv.shape[0], ref.shape[1], ref.shape[3]),
                          dtype=torch.float32, device=qkv.device)
    rows = torch.zeros(batch, dtype=torch.int32, device=qkv.device)  # shape only: not read
    a = make_args(qkv, decay, beta, ref, rows, offsets, out, nk=_nk_from_qkv(qkv, ref),
                  decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps,
                  max_row_len=max_row_len)
    _check(load_library().gdr_fwd_dense(
        ctypes.byref(a), None if initial_state is None else initial_state.data_ptr(),
        None if final is None else final.data_ptr(), _stream(qkv.device)))
    return out, final


def gdr_verify_ring(qkv, decay, beta, state, slot_idx, offsets, ring, ring_slot_idx, out=None, *,
                    decay_is_log=False, use_qk_l2norm=True, scale=0.0, eps=1e-6, max_row_len=0):
    """Verify pass ("gated_delta_recurrence_verify_ring_gpu"); ring is
    [ring_rows, nk, ring_len, record_stride] float32 or bfloat16 (dense)."""
    _dev(ring, "ring", (torch.float32, torch.bfloat16))
    _dev(ring_slot_idx, "ring_slot_idx", torch.int32)
    if ring.dim() != 4 or not ring.is_contiguous():
        raise ValueError("ring must be a contiguous [ring_rows, nk, ring_len, record_stride] tensor")
    if out is None:
        out = torch.empty(gdr_output_shape(qkv.shape[0], state.shape[1], state.shape[3]),
                          dtype=torch.float32, device=qkv.device)
    nk = _nk_from_qkv(qkv, state)
    if ring.shape[1] != nk:
        raise ValueError("ring.shape[1] must equal nk")
    a = make_args(qkv, decay, beta, state, slot_idx, offsets, out, nk=nk, decay_is_log=decay_is_log,
                  use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps, max_row_len=max_row_len)
    _check(load_library().gdr_verify_ring(ctypes.byref(a), ring.data_ptr(), _ring_dtype(ring), ring.shape[0],
                                          ring.shape[2], ring.shape[3], ring_slot_idx.data_ptr(),
                                          _stream(qkv.device)))
    return out


def gdr_fold(state, slot_idx, ring, ring_slot_idx, counts):
    """Fold the first counts[b] records of each row into its slot (in place)."""
    _dev(ring, "ring", (torch.float32, torch.bfloat16))
    _dev(ring_slot_idx, "ring_slot_idx", torch.int32)
    _dev(counts, "counts", torch.int32)
    if ring.dim() != 4 or not ring.is_contiguous():
        raise ValueError("ring must be a contiguous [ring_rows, nk, ring_len, record_stride] tensor")
    a = make_args(None, None, None, state, slot_idx, None, None, nk=ring.shape[1])
    _check(load_library().gdr_fold(ctypes.byref(a), ring.data_ptr(), _ring_dtype(ring), ring.shape[0],
                                   ring.shape[2], ring.shape[3], ring_slot_idx.data_ptr(),
                                   counts.data_ptr(), _stream(state.device)))


def _inter_strides(inter, state):
    if inter.dtype != state.dtype:
        raise TypeError("intermediate_states must have the pool's dtype")
    if inter.dim() != 5 or inter.shape[2:] != state.shape[1:]:
        raise ValueError("intermediate_states must be [slots, n_inter, nv, K, V]")
    if inter.shape[0] < state.shape[0]:
        # the kernels index it by pool slot, which is only checked against the pool's slot count
        raise ValueError(f"intermediate_states has {inter.shape[0]} slot rows; it needs one per pool "
                         f"slot ({state.shape[0]})")
    K, V = state.shape[2:]
    if inter.stride(4) != 1 or inter.stride(3) != V:
        raise ValueError("each [K, V] block of intermediate_states must be dense")
    return inter.stride(0), inter.stride(1), inter.stride(2), inter.shape[1]


def gdr_fwd_snapshots(qkv, decay, beta, state, slot_idx, offsets, inter, steps_per_token, out=None,
                      *, decay_is_log=False, use_qk_l2norm=True, scale=0.0, eps=1e-6,
                      max_row_len=0):
    """Forward pass + snapshots ("core.ssm.ops.gdp.fused_recurrent", intermediate_states)."""
    _dev(inter, "intermediate_states")
    ss, st, sh, n_inter = _inter_strides(inter, state)
    if out is None:
        out = torch.empty(gdr_output_shape(qkv.shape[0], state.shape[1], state.shape[3]),
                          dtype=torch.float32, device=qkv.device)
    a = make_args(qkv, decay, beta, state, slot_idx, offsets, out, nk=_nk_from_qkv(qkv, state),
                  decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps,
                  max_row_len=max_row_len)
    _check(load_library().gdr_fwd_snapshots(ctypes.byref(a), inter.data_ptr(), ss, st, sh,
                                            n_inter, int(steps_per_token), _stream(qkv.device)))
    return out


def gdr_rollback(state, slot_idx, inter, accepted):
    """state[slot] <- intermediate_states[slot, accepted[b]] (in place)."""
    _dev(inter, "intermediate_states")
    _dev(accepted, "accepted", torch.int32)
    ss, st, sh, n_inter = _inter_strides(inter, state)
    a = make_args(None, None, None, state, slot_idx, None, None, nk=1)
    _check(load_library().gdr_rollback(ctypes.byref(a), inter.data_ptr(), ss, st, sh, n_inter,
                                       accepted.data_ptr(), _stream(state.device)))


_DTYPES = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(fn, args, device: int) -> int:
    """fn(args, stream) on a device's current stream; a C entry launches on the
    current device, which is changed around the call where it is another."""
    if device != _current_device():
        with torch.cuda.device(device):
            return fn(args, _stream(device))
    return fn(args, _raw_stream(device) if _raw_stream is not None else _stream(device))


def _tensors(**tensors):
    """Refuses what is no tensor, before anything is asked of it."""
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


def _refuse(device, dtypes, **tensors):
    """Says what is wrong with one of a call's tensors: not one, not on the
    call's device, or not of the wanted dtype (of float32 and bfloat16 where
    dtypes has none for it)."""
    _tensors(**tensors)
    for name, t in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the call on {device}")
        want = dtypes.get(name)
        if want is None and t.dtype not in _DTYPES:
            raise TypeError(f"{name} has dtype {t.dtype}, expected float32 or bfloat16")
        if want is not None and t.dtype != want:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {want}")


def _linattn_values(q, k, v, decay, state, slot_idx, offsets, out, decay_is_log, scale, max_row_len):
    """The values of gdr_linattn_args for a call's tensors (no workspace), checked."""
    try:
        dev, tok = q.device, q.dtype
        td, sd = _DTYPES[tok], _DTYPES[state.dtype]
        good = (q.is_cuda and k.dtype is tok and v.dtype is tok and out.dtype is tok and decay.dtype is torch.float32 and
                slot_idx.dtype is torch.int32 and offsets.dtype is torch.int32 and
                dev == k.device == v.device == decay.device == state.device == slot_idx.device == offsets.device == out.device)
    except (AttributeError, KeyError):
        good = False
    if not good:
        _refuse(getattr(q, "device", None), {"k": getattr(q, "dtype", None), "v": getattr(q, "dtype", None),
                                             "out": getattr(q, "dtype", None), "decay": torch.float32,
                                             "slot_idx": torch.int32, "offsets": torch.int32},
                q=q, k=k, v=v, decay=decay, state=state, slot_idx=slot_idx, offsets=offsets, out=out)
    if state.dim() != 4:
        raise ValueError("state must be [max_slots, nv, K, V]")
    slots, nv, K, V = state.shape
    if q.dim() != 3 or q.shape != k.shape or q.shape[2] != K:
        raise ValueError(f"q and k must both be [T, nk, {K}]")
    T, nk, _ = q.shape
    if v.shape != (T, nv, V) or out.shape != v.shape:
        raise ValueError(f"v and out must be [T, nv, V] = [{T}, {nv}, {V}]")
    if decay.shape != (nv,):
        raise ValueError(f"decay must be [nv] = [{nv}]")
    if slot_idx.dim() != 1 or not slot_idx.is_contiguous():
        raise ValueError("slot_idx must be a contiguous [batch] int32 tensor")
    batch = slot_idx.shape[0]
    if offsets.shape != (batch + 1,) or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous [batch+1] int32 tensor")
    (qt, qh, qc), (kt, kh, kc), (vt, vh, vc), (ot, oh, oc) = q.stride(), k.stride(), v.stride(), out.stride()
    if qc != 1 or kc != 1 or vc != 1 or oc != 1:
        raise ValueError("q, k, v and out must have a unit channel stride")
    ss, sh, sk, sv = state.stride()
    return (batch, nv, nk, K, V, 1 if decay_is_log else 0, td, sd, T, int(max_row_len), q.data_ptr(), qt, qh, k.data_ptr(), kt,
            kh, v.data_ptr(), vt, vh, decay.data_ptr(), decay.stride(0), out.data_ptr(), ot, oh, state.data_ptr(), ss, sh,
            sk, sv, slots, slot_idx.data_ptr(), offsets.data_ptr(), 0, 0, float(scale))


def _linattn_workspace(lib, args: bytes, device, workspace):
    """The arguments with a workspace, the caller's or a new one of the size the call asks for, and that tensor."""
    if workspace is None:
        need = lib.gdr_linattn_workspace_bytes(args)
        if need < 0:
            _check(need)
        if need == 0:
            return args, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _refuse(device, {"workspace": workspace.dtype}, workspace=workspace)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    a = gdr_linattn_args.from_buffer_copy(args)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return bytes(a), workspace


def gdr_linattn_workspace_bytes(q, k, v, decay, state, slot_idx, offsets, *, max_row_len=0) -> int:
    """Workspace bytes gdr_linattn_fwd would use for these tensors (0: none)."""
    n = load_library().gdr_linattn_workspace_bytes(
        _pack_linattn(*_linattn_values(q, k, v, decay, state, slot_idx, offsets, v, False, 0.0, max_row_len)))
    if n < 0:
        _check(n)
    return int(n)


def gdr_linattn_fwd(q, k, v, decay, state, slot_idx, offsets, out=None, *, decay_is_log=False, scale=0.0,
                    max_row_len=0, workspace=None):
    """Decayed linear attention, S <- lambda_h S + k v^T and out = scale S^T q
    per token, over ragged rows and a slot-indexed pool (include/gdr.h,
    gdr_linattn_args); state updated in place; returns out.

    q, k [T, nk, K], v [T, nv, V] of one dtype (bfloat16 or float32), decay
    [nv] float32 (lambda, or ln lambda with decay_is_log), state
    [max_slots, nv, K, V].  max_row_len = 1 is the single-token step; a tight
    bound lets short rows (drafts, last pieces of prompts) take their own form.
    `workspace` is a device tensor to use instead of a new one of
    gdr_linattn_workspace_bytes() bytes."""
    if out is None:
        if not isinstance(v, torch.Tensor):
            _tensors(v=v)
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    args = _pack_linattn(*_linattn_values(q, k, v, decay, state, slot_idx, offsets, out, decay_is_log, scale, max_row_len))
    lib = _lib or load_library()
    if max_row_len != 1:
        args, workspace = _linattn_workspace(lib, args, q.device, workspace)
    rc = _launch(lib.gdr_linattn_fwd, args, q.get_device())
    if rc:
        _check(rc)
    return out


def prepare_linattn_fwd(q, k, v, decay, state, slot_idx, offsets, out, *, decay_is_log=False, scale=0.0,
                        max_row_len=0, workspace=None) -> "Prepared":
    args = _pack_linattn(*_linattn_values(q, k, v, decay, state, slot_idx, offsets, out, decay_is_log, scale, max_row_len))
    lib = load_library()
    args, workspace = _linattn_workspace(lib, args, q.device, workspace)
    return Prepared(lib.gdr_linattn_fwd, gdr_linattn_args.from_buffer_copy(args), (),
                    (q, k, v, decay, state, slot_idx, offsets, out, workspace), q.device)


_ACTIVATIONS = {None: 0, "silu": 1, "sigmoid": 2}


def _activation(name) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError('activation must be None, "silu" or "sigmoid"')
    return _ACTIVATIONS[name]


def _weight(w, D: int, name: str, device):
    if w is None:
        return 0
    if not (isinstance(w, torch.Tensor) and w.dtype is torch.float32 and w.device == device):
        _refuse(device, {name: torch.float32}, **{name: w})
    if w.shape != (D,) or (D > 1 and w.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous [{D}] float32 tensor")
    return w.data_ptr()


def _rows(t, name: str):
    """(seq stride, head stride) of a [T, H, D] or [T, D] tensor."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have a unit channel stride")
    return (st[0], st[1]) if len(st) == 3 else (st[0], 0)


def _float(t, name: str, device) -> int:
    """The gdr_dtype of a float32 or bfloat16 tensor on the call's device."""
    d = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) and t.is_cuda and t.device == device else None
    if d is None:
        _refuse(device, {}, **{name: t})
    return d


def gdr_gate_norm(x, gate, weight=None, out=None, *, eps=1e-6, activation="silu", gate_first=False, centered=False,
                  out_dtype=None):
    """Norm of a recurrence's output times its activated gate, per token and
    head: out = N(x) * act(gate), or N(x * act(gate)) with gate_first
    (include/gdr.h, gdr_norm_args).  x and gate [T, H, D] or [T, D] (gate may
    also be None, or broadcast over the last dimension), float32 or bfloat16;
    weight [D] float32 or None.  Returns out, of x's shape and out_dtype (by
    default the gate's dtype, or x's)."""
    if not (isinstance(x, torch.Tensor) and (gate is None or isinstance(gate, torch.Tensor))):
        _tensors(x=x, gate=gate)
    dev = x.device
    xd, shape = _float(x, "x", dev), x.shape
    if len(shape) not in (2, 3):
        raise ValueError("x must be [T, H, D] or [T, D]")
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or (x if gate is None else gate).dtype, device=dev)
    elif not isinstance(out, torch.Tensor) or out.shape != shape or (out_dtype is not None and out.dtype != out_dtype):
        _tensors(out=out)
        raise ValueError("out must have x's shape and dtype out_dtype")
    od = _float(out, "out", dev)
    T, D = shape[0], shape[-1]
    (xt, xh), (ot, oh) = _rows(x, "x"), _rows(out, "out")
    gp, gd, gt, gh, ge = 0, 0, 0, 0, 0
    if gate is not None:
        gd = _float(gate, "gate", dev)
        if gate.shape != shape and (gate.shape[:-1] != shape[:-1] or gate.shape[-1] != 1):
            raise ValueError("gate must have x's shape, or 1 in its last dimension")
        gp, (gt, gh), ge = gate.data_ptr(), _rows(gate, "gate"), int(gate.shape[-1] == D)
    elif gate_first:
        raise ValueError("gate_first needs a gate")
    args = _pack_norm(T, shape[1] if len(shape) == 3 else 1, D, xd, gd, 0, od, _activation(activation),
                      1 if gate_first else 0, 1, 0, 1 if centered else 0, eps, 1.0, x.data_ptr(), xt, xh, gp, gt, gh, ge,
                      0, 0, 0, 0, 0, 0, out.data_ptr(), ot, oh, _weight(weight, D, "weight", dev), 0)
    rc = _launch((_lib or load_library()).gdr_block_norm, args, x.get_device())
    if rc:
        _check(rc)
    return out


def gdr_residual_norm(block, residual, weight, *, post_weight=None, gate=None, activation=None, residual_scale=1.0,
                      eps=1e-6, centered=False, residual_out=None, out=None, out_dtype=None):
    """Block boundary in one pass: h = residual + residual_scale * act(gate) *
    N(block; post_weight), out = N(h; weight) (include/gdr.h, gdr_norm_args).

    residual [T, D]; block [T, D], or None for the first norm of a stack (out
    = N(residual)); post_weight [D] float32, or None for no norm of the
    block's output; gate [T, D], [T, 1], [D] or None; weight [D] float32, or
    None for a norm without one.  Returns (residual_out, out): residual_out
    may be residual itself (in place) and is residual where block is None;
    out has out_dtype (by default the block's dtype, or residual's)."""
    if not (isinstance(residual, torch.Tensor) and (block is None or isinstance(block, torch.Tensor))):
        _tensors(residual=residual, block=block)
    dev = residual.device
    rd, shape = _float(residual, "residual", dev), residual.shape
    if len(shape) != 2:
        raise ValueError("residual must be [T, D]")
    T, D = shape
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or (residual if block is None else block).dtype, device=dev)
    elif not isinstance(out, torch.Tensor) or out.shape != shape or (out_dtype is not None and out.dtype != out_dtype):
        _tensors(out=out)
        raise ValueError("out must be [T, D] of dtype out_dtype")
    od = _float(out, "out", dev)
    ot, rt = _rows(out, "out")[0], _rows(residual, "residual")[0]
    xp, xd, xt, rop, rot = 0, 0, 0, 0, 0
    if block is None:
        if gate is not None or post_weight is not None or residual_out is not None:
            raise ValueError("gate, post_weight and residual_out need a block")
        h = residual
    else:
        xd = _float(block, "block", dev)
        if block.shape != shape:
            raise ValueError("block must have residual's shape")
        xp, xt = block.data_ptr(), _rows(block, "block")[0]
        h = torch.empty(shape, dtype=residual.dtype, device=dev) if residual_out is None else residual_out
        if h is not residual and (_float(h, "residual_out", dev) != rd or h.shape != shape):
            raise ValueError("residual_out must have residual's shape and dtype")
        rop, rot = h.data_ptr(), _rows(h, "residual_out")[0]
    gp, gd, gt, ge = 0, 0, 0, 0
    if gate is not None:
        gd, gp = _float(gate, "gate", dev), gate.data_ptr()
        if gate.shape == (D,):
            ge = 1
            if D > 1 and gate.stride(0) != 1:
                raise ValueError("gate must have a unit channel stride")
        elif gate.shape in ((T, D), (T, 1)):
            gt, ge = _rows(gate, "gate")[0], int(gate.shape[1] == D)
        else:
            raise ValueError("gate must be [T, D], [T, 1] or [D]")
    args = _pack_norm(T, 1, D, xd, gd, rd, od, _activation(activation), 0, 0 if post_weight is None else 1, 1,
                      1 if centered else 0, eps, residual_scale, xp, xt, 0, gp, gt, 0, ge, residual.data_ptr(), rt, 0,
                      rop, rot, 0, out.data_ptr(), ot, 0, _weight(post_weight, D, "post_weight", dev),
                      _weight(weight, D, "weight", dev))
    rc = _launch((_lib or load_library()).gdr_block_norm, args, residual.get_device())
    if rc:
        _check(rc)
    return h, out


_F32, _I32 = torch.float32, torch.int32


def _ints(t, shape, name: str, device) -> int:
    """The pointer of a contiguous int32 tensor of a call's rows or tokens."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _I32 and t.device == device):
        _refuse(device, {name: _I32}, **{name: t})
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} int32 tensor")
    return t.data_ptr()


def _ragged(slot_idx, offsets, counts, keep_state, state_only, device):
    """(batch, slot_idx, offsets, counts) of a call over ragged rows, as pointers."""
    if not keep_state and (state_only or counts is not None):
        raise ValueError("state_only and counts need keep_state")
    try:
        n, = shape = slot_idx.shape
        if (slot_idx.dtype is _I32 and offsets.dtype is _I32 and slot_idx.device == device == offsets.device and
                offsets.shape == (n + 1,) and slot_idx.is_contiguous() and offsets.is_contiguous()):
            return n, slot_idx.data_ptr(), offsets.data_ptr(), 0 if counts is None else _ints(counts, shape, "counts", device)
    except (AttributeError, TypeError, ValueError):
        pass
    _tensors(slot_idx=slot_idx, offsets=offsets)
    if slot_idx.dim() != 1:
        raise ValueError("slot_idx must be a contiguous [batch] int32 tensor")
    _ints(slot_idx, tuple(slot_idx.shape), "slot_idx", device)
    _ints(offsets, (slot_idx.shape[0] + 1,), "offsets", device)
    return n, slot_idx.data_ptr(), offsets.data_ptr(), 0 if counts is None else _ints(counts, shape, "counts", device)


def _output(out, like, state_only):
    """(tensor, pointer, strides) of a call's output: the caller's, a new one like `like`, or none."""
    if state_only:
        if out is not None:
            raise ValueError("state_only has no out")
        return None, 0, (0,) * like.dim()
    if out is None:
        out = torch.empty_like(like)
    else:
        if not isinstance(out, torch.Tensor):
            _tensors(out=out)
        if out.shape != like.shape or out.dtype != like.dtype or out.device != like.device:
            raise ValueError("out must have x's shape, dtype and device")
    st = out.stride()
    if st[-1] != 1 and out.shape[-1] > 1:
        raise ValueError("out must have a unit channel stride")
    return out, out.data_ptr(), st


def _short_conv_refuse(x, weight, conv_state):
    """Says what is wrong with a convolution's tensors."""
    _tensors(x=x, weight=weight)
    dev = x.device
    _refuse(dev, {"weight": _F32}, x=x, weight=weight)
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be [T, channels] with a unit channel stride")
    if weight.dim() != 2 or weight.shape[0] != x.shape[1]:
        raise ValueError(f"weight must be [channels, width] with {x.shape[1]} channels")
    width = weight.shape[1]
    if width == 1:
        raise ValueError("a convolution of width 1 has no conv_state")
    _refuse(dev, {}, conv_state=conv_state)
    raise ValueError(f"conv_state must be [slots, {x.shape[1]}, {width - 1}]")


def _short_conv_args(x, weight, bias, conv_state, slot_idx, offsets, out, activation, counts, keep_state, state_only, max_row_len):
    """(packed gdr_short_conv_args, out)."""
    sp, sd, ss, sc, st, slots = 0, GDR_F32, 0, 0, 0, 1 << 30
    try:
        dev, td = x.device, _DTYPES[x.dtype]
        (T, C), (xt, xc) = x.shape, x.stride()
        (wc, width), (wsc, wst) = weight.shape, weight.stride()
        good = (xc == 1 or C == 1) and wc == C and weight.dtype is _F32 and weight.device == dev and x.is_cuda
        if width > 1:
            sd = _DTYPES[conv_state.dtype]
            (slots, cc, taps), (ss, sc, st), sp = conv_state.shape, conv_state.stride(), conv_state.data_ptr()
            good = good and cc == C and taps == width - 1 and conv_state.device == dev
        else:
            good = good and conv_state is None
    except (AttributeError, KeyError, ValueError, TypeError):
        good = False
    if not good:
        _short_conv_refuse(x, weight, conv_state)
    if activation is not None and activation != "silu":
        raise ValueError('activation must be "silu" or None')
    n, slot, off, cnt = _ragged(slot_idx, offsets, counts, keep_state, state_only, dev)
    out, op, ost = _output(out, x, state_only)
    return _pack_short_conv(n, C, width, 0 if activation is None else 1, td, sd, 1 if keep_state else 0, T, int(max_row_len),
                            x.data_ptr(), xt, weight.data_ptr(), wsc, wst, _weight(bias, C, "bias", dev), op, ost[0], sp, ss, sc, st,
                            slots, slot, off, cnt), out


def gdr_short_conv(x, weight, bias, conv_state, slot_idx, offsets, out=None, *, activation="silu", counts=None,
                   keep_state=True, state_only=False, max_row_len=0):
    """Short causal depthwise convolution over ragged rows and a slot-indexed
    state pool (include/gdr.h, gdr_short_conv_args); conv_state updated in
    place; returns out.

    x [T, channels] float32 or bfloat16, weight [channels, width] float32 (width
    1 to 4), bias [channels] float32 or None, conv_state [slots, channels,
    width-1] float32 or bfloat16 (None for width 1).  keep_state=False leaves
    the pool as it is (a verify pass of drafts); counts [batch] int32 takes only
    a row's first tokens into its slot; state_only=True computes no output and
    returns None.  max_row_len bounds the rows' lengths (1: single tokens)."""
    args, out = _short_conv_args(x, weight, bias, conv_state, slot_idx, offsets, out, activation, counts, keep_state,
                                 state_only, max_row_len)
    rc = _launch((_lib or load_library()).gdr_short_conv, args, x.get_device())
    if rc:
        _check(rc)
    return out


def prepare_short_conv(x, weight, bias, conv_state, slot_idx, offsets, out, *, activation="silu", counts=None,
                       keep_state=True, state_only=False, max_row_len=0) -> "Prepared":
    if out is None and not state_only:
        raise ValueError("a prepared call needs its out")
    args, out = _short_conv_args(x, weight, bias, conv_state, slot_idx, offsets, out, activation, counts, keep_state,
                                 state_only, max_row_len)
    return Prepared(load_library().gdr_short_conv, gdr_short_conv_args.from_buffer_copy(args), (),
                    (x, weight, bias, conv_state, slot_idx, offsets, out, counts), x.device)


_NO2 = (0, 0)


def _per_channel(t, shape, name: str, device):
    """(pointer, strides) of a float32 tensor of a layer's channels; broadcast dimensions as strides of 0."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _F32 and t.device == device):
        _refuse(device, {name: _F32}, **{name: t})
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (expand what it shares)")
    return t.data_ptr(), t.stride()


def _scan_refuse(x, dt, B, C, z, state):
    """Says what is wrong with the tokens' tensors of a scan."""
    _tensors(x=x, dt=dt, state=state, B=B, C=C)
    dev, want = x.device, {"B": x.dtype, "C": x.dtype, "z": x.dtype}
    _refuse(dev, want, x=x, dt=dt, state=state, B=B, C=C, **({} if z is None else {"z": z}))
    if state.dim() != 4:
        raise ValueError("state must be [max_slots, nv, K, V]")
    _, nv, K, V = state.shape
    if x.dim() != 3 or x.shape[1:] != (nv, V):
        raise ValueError(f"x must be [T, nv, V] = [T, {nv}, {V}]")
    if dt.shape != x.shape:
        raise ValueError("dt must have x's shape (expand what it shares)")
    if B.dim() != 3 or B.shape != C.shape or B.shape[0] != x.shape[0] or B.shape[2] != K or (K > 1 and (B.stride(2), C.stride(2)) != (1, 1)):
        raise ValueError(f"B and C must both be [T, nk, K] = [{x.shape[0]}, nk, {K}] with a unit stride along K")
    if z is not None and (z.shape != x.shape or (V > 1 and z.stride(2) != 1)):
        raise ValueError("z must have x's shape and a unit channel stride")
    raise ValueError("x must have a unit channel stride, and dt one or one value a head")


def _scan_args(x, dt, A, B, C, state, slot_idx, offsets, out, D, z, dt_bias, dt_softplus, counts, keep_state, state_only,
               max_row_len):
    """(packed gdr_scan_args without a workspace, out)."""
    zp, zt, zh = 0, 0, 0
    try:
        dev, tok, shape, bshape = x.device, x.dtype, x.shape, B.shape
        td, dd, sd = _DTYPES[tok], _DTYPES[dt.dtype], _DTYPES[state.dtype]
        slots, nv, K, V = state.shape
        T, xn, xv = shape
        (xt, xh, xc), (tt, th, te), (Bt, Bh, Bk), (Ct, Ch, Ck) = x.stride(), dt.stride(), B.stride(), C.stride()
        good = (x.is_cuda and B.dtype is tok and C.dtype is tok and dev == dt.device == B.device == C.device == state.device and
                xn == nv and xv == V and shape == dt.shape and bshape[0] == T and bshape[2] == K and bshape == C.shape and
                (V == 1 or (xc == 1 and (te == 1 or te == 0))) and (K == 1 or (Bk == 1 and Ck == 1)))
        if z is not None:
            zt, zh, zc = z.stride()
            zp = z.data_ptr()
            good = good and z.dtype is tok and z.device == dev and z.shape == shape and (zc == 1 or V == 1)
    except (AttributeError, KeyError, ValueError, TypeError, IndexError):
        good = False
    if not good:
        _scan_refuse(x, dt, B, C, z, state)
    ap, (ah, ak, av) = _per_channel(A, (nv, K, V), "A", dev)
    dp, (dh, dv) = (0, _NO2) if D is None else _per_channel(D, (nv, V), "D", dev)
    bp, (bh, bv) = (0, _NO2) if dt_bias is None else _per_channel(dt_bias, (nv, V), "dt_bias", dev)
    n, slot, off, cnt = _ragged(slot_idx, offsets, counts, keep_state, state_only, dev)
    out, op, (ot, oh, _) = _output(out, x, state_only)
    ss, sh, sk, sv = state.stride()
    return _pack_scan(n, nv, bshape[1], K, V, 1 if dt_softplus else 0, td, dd, sd, 1 if keep_state else 0, T, int(max_row_len),
                      x.data_ptr(), xt, xh, dt.data_ptr(), tt, th, te if V > 1 else 1, B.data_ptr(), Bt, Bh, C.data_ptr(), Ct,
                      Ch, zp, zt, zh, ap, ah, ak, av, dp, dh, dv, bp, bh, bv, op, ot, oh, state.data_ptr(), ss, sh, sk, sv, slots,
                      slot, off, cnt, 0, 0), out


def _scan_workspace(lib, args: bytes, device, workspace):
    """The arguments with a workspace, the caller's or a new one of the size the call asks for, and that tensor."""
    if workspace is None:
        need = lib.gdr_selective_scan_workspace_bytes(args)
        if need < 0:
            _check(need)
        if need == 0:
            return args, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _refuse(device, {"workspace": getattr(workspace, "dtype", None)}, workspace=workspace)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    a = gdr_scan_args.from_buffer_copy(args)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return bytes(a), workspace


def gdr_selective_scan_workspace_bytes(x, dt, A, B, C, state, slot_idx, offsets, *, max_row_len=0) -> int:
    """Workspace bytes gdr_selective_scan would use for these tensors (0: none)."""
    args, _ = _scan_args(x, dt, A, B, C, state, slot_idx, offsets, x, None, None, None, True, None, True, False, max_row_len)
    n = load_library().gdr_selective_scan_workspace_bytes(args)
    if n < 0:
        _check(n)
    return int(n)


def gdr_selective_scan(x, dt, A, B, C, state, slot_idx, offsets, out=None, *, D=None, z=None, dt_bias=None, dt_softplus=True,
                       counts=None, keep_state=True, state_only=False, max_row_len=0, workspace=None):
    """Selective state space scan over ragged rows and a slot-indexed pool
    (include/gdr.h, gdr_scan_args): per token d = softplus(dt + dt_bias), S <-
    exp(d A) S + d x B, out = (C S + D x) silu(z); state updated in place;
    returns out.

    x, z [T, nv, V] and B, C [T, nk, K] of one dtype (bfloat16 or float32), dt [T,
    nv, V] of that dtype or float32 (or one value a head, expanded), A [nv, K,
    V], D and dt_bias [nv, V] float32 (expanded where shared), state [max_slots,
    nv, K, V] bfloat16 or float32.  keep_state=False leaves the pool as it is (a
    verify pass of drafts); counts [batch] int32 takes only a row's first tokens
    into its slot; state_only=True computes no output and returns None.
    max_row_len bounds the rows' lengths (1: single tokens).  `workspace` is a
    device tensor to use instead of a new one of
    gdr_selective_scan_workspace_bytes() bytes."""
    args, out = _scan_args(x, dt, A, B, C, state, slot_idx, offsets, out, D, z, dt_bias, dt_softplus, counts, keep_state,
                           state_only, max_row_len)
    lib = _lib or load_library()
    if workspace is not None or not 1 <= max_row_len <= 16:  # rows so short are never cut
        args, workspace = _scan_workspace(lib, args, x.device, workspace)
    rc = _launch(lib.gdr_selective_scan, args, x.get_device())
    if rc:
        _check(rc)
    return out


def prepare_selective_scan(x, dt, A, B, C, state, slot_idx, offsets, out, *, D=None, z=None, dt_bias=None, dt_softplus=True,
                           counts=None, keep_state=True, state_only=False, max_row_len=0, workspace=None) -> "Prepared":
    if out is None and not state_only:
        raise ValueError("a prepared call needs its out")
    args, out = _scan_args(x, dt, A, B, C, state, slot_idx, offsets, out, D, z, dt_bias, dt_softplus, counts, keep_state,
                           state_only, max_row_len)
    lib = load_library()
    args, workspace = _scan_workspace(lib, args, x.device, workspace)
    return Prepared(lib.gdr_selective_scan, gdr_scan_args.from_buffer_copy(args), (),
                    (x, dt, A, B, C, state, slot_idx, offsets, out, D, z, dt_bias, counts, workspace), x.device)


def _accept_refuse(target, draft, tokens, offsets, uniforms, row_uniforms):
    """Says what is wrong with a verification's tensors."""
    _tensors(target=target, tokens=tokens, offsets=offsets, uniforms=uniforms, row_uniforms=row_uniforms)
    dev = target.device
    want = {"draft": target.dtype, "tokens": _I32, "offsets": _I32, "uniforms": _F32, "row_uniforms": _F32}
    _refuse(dev, want, target=target, tokens=tokens, offsets=offsets, uniforms=uniforms, row_uniforms=row_uniforms,
            **({} if draft is None else {"draft": draft}))
    if target.dim() != 2 or (target.shape[1] > 1 and target.stride(1) != 1):
        raise ValueError("target must be [T, vocab] with a unit stride along the vocabulary")
    if draft is not None and (draft.shape != target.shape or (target.shape[1] > 1 and draft.stride(1) != 1)):
        raise ValueError("draft must have target's shape and a unit stride along the vocabulary")
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be a contiguous [batch+1] int32 tensor")
    T, n = target.shape[0], offsets.shape[0] - 1
    for name, t, size in (("tokens", tokens, T), ("uniforms", uniforms, T), ("row_uniforms", row_uniforms, n), ("offsets", offsets, n + 1)):
        if t.shape != (size,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [{size}] tensor")
    raise ValueError("the tensors of the call do not fit together")


def _accept_args(target, draft, tokens, offsets, uniforms, row_uniforms, max_row_len, out, counts):
    """(packed gdr_accept_args, out, counts)."""
    qp, qt = 0, 0
    try:
        dev, pd = target.device, _DTYPES[target.dtype]
        (T, vocab), (pt, pc) = shape, _ = target.shape, target.stride()
        rows, = offsets.shape
        good = (target.is_cuda and (pc == 1 or vocab == 1) and rows >= 1 and tokens.dtype is _I32 and offsets.dtype is _I32 and
                uniforms.dtype is _F32 and row_uniforms.dtype is _F32 and
                dev == tokens.device == offsets.device == uniforms.device == row_uniforms.device and
                tokens.shape == (T,) == uniforms.shape and row_uniforms.shape == (rows - 1,) and tokens.is_contiguous() and
                offsets.is_contiguous() and uniforms.is_contiguous() and row_uniforms.is_contiguous())
        if draft is not None:
            (qt, qc), qp = draft.stride(), draft.data_ptr()
            good = good and draft.dtype is target.dtype and draft.device == dev and draft.shape == shape and (qc == 1 or vocab == 1)
    except (AttributeError, KeyError, ValueError, TypeError):
        good = False
    if not good:
        _accept_refuse(target, draft, tokens, offsets, uniforms, row_uniforms)
    n, width = rows - 1, int(max_row_len)
    if width < 1:
        raise ValueError("max_row_len must be at least 1 (it is the width of the returned tokens)")
    if out is None:
        out, ot = torch.empty((n, width), dtype=_I32, device=dev), width
    else:
        if not (isinstance(out, torch.Tensor) and out.dtype is _I32 and out.device == dev):
            _refuse(dev, {"out": _I32}, out=out)
        if out.shape != (n, width) or (width > 1 and out.stride(1) != 1):
            raise ValueError(f"out must be [{n}, {width}] with a unit stride along a row")
        ot = out.stride(0)
    if counts is None:
        counts = torch.empty(n, dtype=_I32, device=dev)
        cp = counts.data_ptr()
    else:
        cp = _ints(counts, (n,), "counts", dev)
    return _pack_accept(n, vocab, pd, width, T, target.data_ptr(), pt, qp, qt, tokens.data_ptr(), offsets.data_ptr(),
                        uniforms.data_ptr(), row_uniforms.data_ptr(), out.data_ptr(), ot, cp), out, counts


def gdr_accept_drafts(target, draft, tokens, offsets, uniforms, row_uniforms, *, max_row_len, out=None, counts=None):
    """Verification of drafted tokens by rejection (include/gdr.h,
    gdr_accept_args): which of each row's drafts the target's probabilities let
    through, and the token drawn behind them.  Returns (out, counts): out
    [batch, max_row_len] int32 has each row's accepted drafts, the drawn token and
    -1 behind it; counts [batch] int32 is their number, what gdr_fold and the
    counts arguments of the state_only calls take (gdr_rollback: counts - 1).

    target and draft [T, vocab] float32 or bfloat16 probabilities of what follows
    each token (draft None: the drafts were not drawn from probabilities),
    tokens [T] int32 (each row's last known token and its drafts), offsets
    [batch+1] int32, uniforms [T] and row_uniforms [batch] float32 in [0, 1)."""
    args, out, counts = _accept_args(target, draft, tokens, offsets, uniforms, row_uniforms, max_row_len, out, counts)
    rc = _launch((_lib or load_library()).gdr_accept_drafts, args, target.get_device())
    if rc:
        _check(rc)
    return out, counts


def prepare_accept_drafts(target, draft, tokens, offsets, uniforms, row_uniforms, out, counts, *, max_row_len) -> "Prepared":
    if out is None or counts is None:
        raise ValueError("a prepared call needs its out and counts")
    args, out, counts = _accept_args(target, draft, tokens, offsets, uniforms, row_uniforms, max_row_len, out, counts)
    return Prepared(load_library().gdr_accept_drafts, gdr_accept_args.from_buffer_copy(args), (),
                    (target, draft, tokens, offsets, uniforms, row_uniforms, out, counts), target.device)


def gdr_get_status(clear: bool = True) -> int:
    """Device status word (GDR_STATUS_* bits); synchronises the device."""
    v = ctypes.c_uint32(0)
    _check(load_library().gdr_get_status(ctypes.byref(v), int(bool(clear))))
    return int(v.value)


def gdr_probe_fma(pattern: int, warps_per_subpartition: int, iterations: int, sink: torch.Tensor) -> int:
    """Diagnostic FP32-pipe probe of include/gdr.h (pattern 0: the recurrence's
    per-element sweep; 1: packed FMAs with reusable operands; 2: with three
    distinct operands).  Launches on the current stream; returns the CTA count
    (one per SM, 128 * warps_per_subpartition threads each)."""
    _dev(sink, "sink", torch.float32)
    if not sink.is_contiguous():
        raise ValueError("sink must be contiguous")
    ctas = ctypes.c_int32(0)
    _check(load_library().gdr_probe_fma(int(pattern), int(warps_per_subpartition), int(iterations), sink.data_ptr(),
                                        sink.numel(), ctypes.byref(ctas), _stream(sink.device)))
    return int(ctas.value)


def status_names(bits: int):
    return [n for b, n in STATUS_BITS.items() if bits & b]


class Prepared:
    """A C-ABI call with its arguments marshalled once.

    Calling it re-issues the same entry point on the same device buffers with
    no per-call Python marshalling (the buffers' contents may change between
    calls; their addresses, shapes and strides may not).  Useful for repeated
    decode steps and for capturing the call into a CUDA graph."""

    def __init__(self, fn, args: gdr_step_args, extra, keep, device):
        self._fn = fn
        self._args = args
        self._extra = extra
        self._keep = keep  # tensors whose storage the call uses
        self._device = device

    def __call__(self, stream: Optional[int] = None):
        s = _stream(self._device) if stream is None else stream
        if self._device.index not in (None, _current_device()):  # a C entry launches on the current device
            with torch.cuda.device(self._device):
                return _check(self._fn(ctypes.byref(self._args), *self._extra, s))
        _check(self._fn(ctypes.byref(self._args), *self._extra, s))


def prepare_fwd(qkv, decay, beta, state, slot_idx, offsets, out, *, decay_is_log=False,
                use_qk_l2norm=True, scale=0.0, eps=1e-6, max_row_len=0) -> Prepared:
    a = make_args(qkv, decay, beta, state, slot_idx, offsets, out, nk=_nk_from_qkv(qkv, state),
                  decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps,
                  max_row_len=max_row_len)
    return Prepared(load_library().gdr_fwd, a, (),
                    (qkv, decay, beta, state, slot_idx, offsets, out), qkv.device)


def prepare_verify_ring(qkv, decay, beta, state, slot_idx, offsets, ring, ring_slot_idx, out, *,
                        decay_is_log=False, use_qk_l2norm=True, scale=0.0, eps=1e-6,
                        max_row_len=0) -> Prepared:
    _dev(ring, "ring", (torch.float32, torch.bfloat16))
    _dev(ring_slot_idx, "ring_slot_idx", torch.int32)
    if ring.dim() != 4 or not ring.is_contiguous():
        raise ValueError("ring must be a contiguous [ring_rows, nk, ring_len, record_stride] tensor")
    a = make_args(qkv, decay, beta, state, slot_idx, offsets, out, nk=_nk_from_qkv(qkv, state),
                  decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps,
                  max_row_len=max_row_len)
    extra = (ring.data_ptr(), _ring_dtype(ring), ring.shape[0], ring.shape[2], ring.shape[3],
             ring_slot_idx.data_ptr())
    return Prepared(load_library().gdr_verify_ring, a, extra,
                    (qkv, decay, beta, state, slot_idx, offsets, out, ring, ring_slot_idx),
                    qkv.device)


def prepare_fold(state, slot_idx, ring, ring_slot_idx, counts) -> Prepared:
    _dev(ring, "ring", (torch.float32, torch.bfloat16))
    _dev(ring_slot_idx, "ring_slot_idx", torch.int32)
    _dev(counts, "counts", torch.int32)
    if ring.dim() != 4 or not ring.is_contiguous():
        raise ValueError("ring must be a contiguous [ring_rows, nk, ring_len, record_stride] tensor")
    a = make_args(None, None, None, state, slot_idx, None, None, nk=ring.shape[1])
    extra = (ring.data_ptr(), _ring_dtype(ring), ring.shape[0], ring.shape[2], ring.shape[3],
             ring_slot_idx.data_ptr(), counts.data_ptr())
    return Prepared(load_library().gdr_fold, a, extra,
                    (state, slot_idx, ring, ring_slot_idx, counts), state.device)


def prepare_fwd_snapshots(qkv, decay, beta, state, slot_idx, offsets, inter, steps_per_token, out,
                          *, decay_is_log=False, use_qk_l2norm=True, scale=0.0, eps=1e-6,
                          max_row_len=0) -> Prepared:
    _dev(inter, "intermediate_states")
    ss, st, sh, n_inter = _inter_strides(inter, state)
    a = make_args(qkv, decay, beta, state, slot_idx, offsets, out, nk=_nk_from_qkv(qkv, state),
                  decay_is_log=decay_is_log, use_qk_l2norm=use_qk_l2norm, scale=scale, eps=eps,
                  max_row_len=max_row_len)
    extra = (inter.data_ptr(), ss, st, sh, n_inter, int(steps_per_token))
    return Prepared(load_library().gdr_fwd_snapshots, a, extra,
                    (qkv, decay, beta, state, slot_idx, offsets, out, inter), qkv.device)


def prepare_rollback(state, slot_idx, inter, accepted) -> Prepared:
    _dev(inter, "intermediate_states")
    _dev(accepted, "accepted", torch.int32)
    ss, st, sh, n_inter = _inter_strides(inter, state)
    a = make_args(None, None, None, state, slot_idx, None, None, nk=1)
    extra = (inter.data_ptr(), ss, st, sh, n_inter, accepted.data_ptr())
    return Prepared(load_library().gdr_rollback, a, extra, (state, slot_idx, inter, accepted),
                    state.device)
