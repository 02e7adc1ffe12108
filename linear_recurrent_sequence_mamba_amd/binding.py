"""ctypes binding of libm3ssm (include/m3ssm.h).

The functions carry the C names and only marshal arguments: they check that
the torch tensors match the dims (shape, dtype, device, contiguity) so that
no kernel can be handed a buffer smaller than it will touch, then pass the
raw device pointers and the current HIP stream to the library.  All compute
runs in the library's HIP kernels; there is no fallback path.  If the shared
library is missing the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libm3ssm.so")

M3_F32, M3_BF16 = 0, 1
M3_THETA_IS_ANGLE = 1 << 0
M3_A_PER_TOKEN = 1 << 1
M3_ROPE_HALF = 1 << 0
M3_GATED_CHUNK = 128
M3_DELTA_CHUNK = 64
M3_GATE_SIGMOID, M3_GATE_SILU, M3_BLOCK_RAW = 1 << 0, 1 << 1, 1 << 2

STATUS = {0: "M3_OK", 1: "M3_ERR_NULL", 2: "M3_ERR_SHAPE", 3: "M3_ERR_DTYPE",
          4: "M3_ERR_UNSUPPORTED", 5: "M3_ERR_ALIGN", 6: "M3_ERR_WORKSPACE", 7: "M3_ERR_HIP",
          8: "M3_ERR_TOO_LARGE"}
M3_NOALLOC_SCRATCH_BYTES = 64 << 20


class m3_bc_prep(ctypes.Structure):
    _fields_ = [("B_weight", ctypes.c_void_p), ("C_weight", ctypes.c_void_p),
                ("B_bias", ctypes.c_void_p), ("C_bias", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("rms", ctypes.c_int32)]


class m3_theta_proj(ctypes.Structure):
    _fields_ = [("u", ctypes.c_void_p), ("W", ctypes.c_void_p), ("dim", ctypes.c_int32)]


class m3_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("nheads", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("ngroups", ctypes.c_int32), ("bc", ctypes.POINTER(m3_bc_prep)),
                ("tp", ctypes.POINTER(m3_theta_proj))]


class m3_gated_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("width", ctypes.c_int32), ("dtype", ctypes.c_int32), ("c", ctypes.c_float),
                ("ld_x", ctypes.c_int64), ("ld_r", ctypes.c_int64), ("ld_i", ctypes.c_int64),
                ("ld_g", ctypes.c_int64)]


class m3_qk_dims(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("nheads_q", ctypes.c_int32),
                ("nheads_k", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("eps", ctypes.c_float), ("base", ctypes.c_double),
                ("ld_q", ctypes.c_int64), ("ld_k", ctypes.c_int64), ("ld_dq", ctypes.c_int64),
                ("ld_dk", ctypes.c_int64)]


class m3_delta_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("nheads_k", ctypes.c_int32), ("nheads_v", ctypes.c_int32),
                ("headdim_k", ctypes.c_int32), ("headdim_v", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("ld_q", ctypes.c_int64),
                ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64), ("ld_g", ctypes.c_int64),
                ("ld_beta", ctypes.c_int64)]


class m3_block_dims(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("width", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("eps", ctypes.c_float),
                ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64), ("ld_gate", ctypes.c_int64)]


class m3_attn_dims(ctypes.Structure):
    _fields_ = [("nseq", ctypes.c_int32), ("tokens_q", ctypes.c_int32),
                ("tokens_k", ctypes.c_int32), ("nheads_q", ctypes.c_int32),
                ("nheads_k", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("ld_q", ctypes.c_int64),
                ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64), ("ld_o", ctypes.c_int64),
                ("ld_do", ctypes.c_int64), ("stride_k", ctypes.c_int64),
                ("stride_v", ctypes.c_int64)]


class BCPrep:
    """The in-kernel preparation of B and C (m3_bc_prep): RMS normalisation
    over N per rank column, weight [N] and per-head bias [H, N, R], all fp32
    device tensors or None."""

    def __init__(self, B_weight=None, C_weight=None, B_bias=None, C_bias=None, eps=1e-6,
                 rms=True):
        self.B_weight, self.C_weight = B_weight, C_weight
        self.B_bias, self.C_bias = B_bias, C_bias
        self.eps, self.rms = float(eps), bool(rms)

    def struct(self) -> m3_bc_prep:
        return m3_bc_prep(_ptr(self.B_weight), _ptr(self.C_weight), _ptr(self.B_bias),
                          _ptr(self.C_bias), self.eps, int(self.rms))

    def check(self, H, N, R):
        for name in ("B_weight", "C_weight"):
            _check(name, getattr(self, name), (N,), torch.float32, optional=True)
        for name in ("B_bias", "C_bias"):
            _check(name, getattr(self, name), (H, N, R), torch.float32, optional=True)


class ThetaProj:
    """The in-kernel angle projection (m3_theta_proj): theta = W u per token
    row and head group; u [rows..., D] and W [G, N/2, D] device tensors in
    the input dtype."""

    def __init__(self, u, W):
        self.u, self.W = u, W
        self.dim = int(W.shape[-1])

    def struct(self) -> m3_theta_proj:
        return m3_theta_proj(_ptr(self.u), _ptr(self.W), self.dim)

    def check(self, rows, G, N, dtype):
        _check("tp.u", self.u, tuple(rows) + (self.dim,), dtype)
        _check("tp.W", self.W, (G, N // 2, self.dim), dtype)


class M3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)} ({_status_str(status)})"
        if status == 7:
            msg += f", hip error {_lib().m3_last_hip_error()}"
        super().__init__(msg)


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m linear_recurrent_sequence_mamba_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        vp, sz, dp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(m3_dims)
        lib.m3_prefill_workspace_size.restype = sz
        lib.m3_prefill_workspace_size.argtypes = [dp]
        lib.m3_scan_prefill.restype = ctypes.c_int
        lib.m3_scan_prefill.argtypes = [dp] + [vp] * 13 + [sz, vp]
        lib.m3_scan_prefill_noalloc.restype = ctypes.c_int
        lib.m3_scan_prefill_noalloc.argtypes = [dp] + [vp] * 12 + [vp]
        lib.m3_prefill_backward_workspace_size.restype = sz
        lib.m3_prefill_backward_workspace_size.argtypes = [dp]
        lib.m3_scan_prefill_backward.restype = ctypes.c_int
        lib.m3_scan_prefill_backward.argtypes = [dp] + [vp] * 23 + [sz, vp]
        lib.m3_prefill_varlen_workspace_size.restype = sz
        lib.m3_prefill_varlen_workspace_size.argtypes = [dp]
        lib.m3_scan_prefill_varlen.restype = ctypes.c_int
        lib.m3_scan_prefill_varlen.argtypes = [dp] + [vp] * 14 + [sz, vp]
        lib.m3_decode_step.restype = ctypes.c_int
        lib.m3_decode_step.argtypes = [dp] + [vp] * 11 + [vp]
        lib.m3_decode_tokens.restype = ctypes.c_int
        lib.m3_decode_tokens.argtypes = [dp] + [vp] * 11 + [vp]
        gp, qp, ap, i32 = (ctypes.POINTER(m3_gated_dims), ctypes.POINTER(m3_qk_dims),
                           ctypes.POINTER(m3_attn_dims), ctypes.c_int)
        bp, ep = ctypes.POINTER(m3_block_dims), ctypes.POINTER(m3_delta_dims)
        for name, args in (
                ("m3_gated_scan_workspace_size", [gp, i32]),
                ("m3_gated_scan_backward_workspace_size", [gp, i32]),
                ("m3_qk_norm_rope_backward_workspace_size", [qp]),
                ("m3_delta_scan_workspace_size", [ep, i32]),
                ("m3_delta_scan_backward_workspace_size", [ep, i32]),
                ("m3_block_norm_backward_workspace_size", [bp]),
                ("m3_attn_prefill_varlen_workspace_size", [ap]),
                ("m3_attn_prefill_varlen_backward_workspace_size", [ap]),
                ("m3_attn_decode_workspace_size", [ap])):
            getattr(lib, name).restype = sz
            getattr(lib, name).argtypes = args
        for name, args in (
                ("m3_gated_scan", [gp] + [vp] * 10 + [sz, vp]),
                ("m3_gated_scan_backward", [gp] + [vp] * 15 + [sz, vp]),
                ("m3_gated_step", [gp] + [vp] * 7),
                ("m3_qk_norm_rope", [qp] + [vp] * 8),
                ("m3_qk_norm_rope_backward", [qp] + [vp] * 12 + [sz, vp]),
                ("m3_delta_scan", [ep] + [vp] * 11 + [sz, vp]),
                ("m3_delta_scan_backward", [ep] + [vp] * 16 + [sz, vp]),
                ("m3_delta_step", [ep] + [vp] * 8),
                ("m3_block_norm", [bp] + [vp] * 9),
                ("m3_block_norm_backward", [bp] + [vp] * 15 + [sz, vp]),
                ("m3_attn_prefill_varlen", [ap] + [vp] * 8 + [sz, vp]),
                ("m3_attn_prefill_varlen_backward", [ap] + [vp] * 12 + [sz, vp]),
                ("m3_attn_decode", [ap] + [vp] * 7 + [sz, vp])):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = args
        lib.m3_status_str.restype = ctypes.c_char_p
        lib.m3_status_str.argtypes = [ctypes.c_int]
        lib.m3_last_hip_error.restype = ctypes.c_int
        lib.m3_last_hip_error.argtypes = []
        _LIB = lib
    return _LIB


def library():
    """The loaded ctypes library (loads it on first use)."""
    return _lib()


def _status_str(s: int) -> str:
    return _lib().m3_status_str(int(s)).decode()


def m3_status_str(status: int) -> str:
    return _status_str(status)


def make_dims(batch, seqlen, nheads, headdim, dstate, rank=1, chunk=0,
              in_dtype=M3_BF16, out_dtype=M3_F32, flags=0, ngroups=0, bc=None,
              tp=None) -> m3_dims:
    """bc: a BCPrep, tp: a ThetaProj (both kept alive by the returned dims)
    or None."""
    d = m3_dims(batch, seqlen, nheads, headdim, dstate, rank, chunk, in_dtype,
                out_dtype, flags, ngroups)
    if bc is not None:
        d._bc_struct = bc.struct()
        d._bc = bc
        d.bc = ctypes.pointer(d._bc_struct)
    if tp is not None:
        d._tp_struct = tp.struct()
        d._tp = tp
        d.tp = ctypes.pointer(d._tp_struct)
    return d


def _check_bc(d: m3_dims):
    bc = getattr(d, "_bc", None)
    if bc is not None:
        bc.check(d.nheads, d.dstate, d.rank)


def _proj(d: m3_dims):
    """The dims' ThetaProj, or None (theta is then a required input)."""
    return getattr(d, "_tp", None)


def groups(d: m3_dims) -> int:
    """B, C and theta groups of a call (ngroups, or nheads when it is 0)."""
    return d.ngroups if d.ngroups > 0 else d.nheads


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return M3_BF16
    if t == torch.float32:
        return M3_F32
    raise TypeError(f"unsupported dtype {t}")


_TORCH = {M3_BF16: torch.bfloat16, M3_F32: torch.float32}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(name, t, shape, dtype, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def m3_prefill_workspace_size(dims: m3_dims) -> int:
    return int(_lib().m3_prefill_workspace_size(ctypes.byref(dims)))


def m3_scan_prefill(dims: m3_dims, x, dt, A, lam, theta, B, C, h0, x_prev, B_prev,
                    y, hT, ws, stream=None) -> None:
    d = dims
    ti, to = _TORCH.get(d.in_dtype), _TORCH.get(d.out_dtype)
    if ti is not None and to is not None:
        Bsz, T, H, P, N, R = d.batch, d.seqlen, d.nheads, d.headdim, d.dstate, d.rank
        G = groups(d)
        _check("x", x, (Bsz, T, H, P, R), ti)
        _check("dt", dt, (Bsz, T, H), ti)
        _check("A", A, (Bsz, T, H) if d.flags & M3_A_PER_TOKEN else (H,), torch.float32)
        _check("lam", lam, (Bsz, T, H), ti)
        _check("theta", theta, (Bsz, T, G, N // 2), ti, optional=_proj(d) is not None)
        if _proj(d) is not None:
            _proj(d).check((Bsz, T), G, N, ti)
        _check("B", B, (Bsz, T, G, N, R), ti)
        _check("C", C, (Bsz, T, G, N, R), ti)
        _check("h0", h0, (Bsz, H, P, N), torch.float32, optional=True)
        _check("x_prev", x_prev, (Bsz, H, P, R), ti, optional=True)
        _check("B_prev", B_prev, (Bsz, G, N, R), ti, optional=True)
        _check("y", y, (Bsz, T, H, P, R), to)
        _check("hT", hT, (Bsz, H, P, N), torch.float32, optional=True)
    nbytes = 0
    if ws is not None:
        if not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous device tensor")
        nbytes = ws.numel() * ws.element_size()
    _check_bc(d)
    st = _lib().m3_scan_prefill(ctypes.byref(d), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam),
                                _ptr(theta), _ptr(B), _ptr(C), _ptr(h0), _ptr(x_prev),
                                _ptr(B_prev), _ptr(y), _ptr(hT), _ptr(ws), nbytes,
                                _stream(stream))
    if st != 0:
        raise M3Error(st, "m3_scan_prefill")


def m3_scan_prefill_noalloc(dims: m3_dims, x, dt, A, lam, theta, B, C, h0, x_prev, B_prev,
                            y, hT, stream=None) -> None:
    """m3_scan_prefill with the library's own scratch buffer (no workspace
    argument; calls that overlap on one GPU race)."""
    d = dims
    ti, to = _TORCH.get(d.in_dtype), _TORCH.get(d.out_dtype)
    if ti is not None and to is not None:
        Bsz, T, H, P, N, R = d.batch, d.seqlen, d.nheads, d.headdim, d.dstate, d.rank
        G = groups(d)
        _check("x", x, (Bsz, T, H, P, R), ti)
        _check("dt", dt, (Bsz, T, H), ti)
        _check("A", A, (Bsz, T, H) if d.flags & M3_A_PER_TOKEN else (H,), torch.float32)
        _check("lam", lam, (Bsz, T, H), ti)
        _check("theta", theta, (Bsz, T, G, N // 2), ti, optional=_proj(d) is not None)
        if _proj(d) is not None:
            _proj(d).check((Bsz, T), G, N, ti)
        _check("B", B, (Bsz, T, G, N, R), ti)
        _check("C", C, (Bsz, T, G, N, R), ti)
        _check("h0", h0, (Bsz, H, P, N), torch.float32, optional=True)
        _check("x_prev", x_prev, (Bsz, H, P, R), ti, optional=True)
        _check("B_prev", B_prev, (Bsz, G, N, R), ti, optional=True)
        _check("y", y, (Bsz, T, H, P, R), to)
        _check("hT", hT, (Bsz, H, P, N), torch.float32, optional=True)
    _check_bc(d)
    st = _lib().m3_scan_prefill_noalloc(ctypes.byref(d), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam),
                                        _ptr(theta), _ptr(B), _ptr(C), _ptr(h0), _ptr(x_prev),
                                        _ptr(B_prev), _ptr(y), _ptr(hT), _stream(stream))
    if st != 0:
        raise M3Error(st, "m3_scan_prefill_noalloc")


def m3_prefill_backward_workspace_size(dims: m3_dims) -> int:
    return int(_lib().m3_prefill_backward_workspace_size(ctypes.byref(dims)))


GRAD_NAMES = ("x", "dt", "A", "lam", "theta", "B", "C", "h0", "x_prev", "B_prev")


def m3_scan_prefill_backward(dims: m3_dims, x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, dy,
                             dhT, grads: dict, ws, stream=None) -> None:
    """grads: fp32 device tensors keyed by GRAD_NAMES (h0, x_prev, B_prev may
    be missing or None)."""
    d = dims
    ti, to = _TORCH.get(d.in_dtype), _TORCH.get(d.out_dtype)
    if ti is not None and to is not None:
        Bsz, T, H, P, N, R = d.batch, d.seqlen, d.nheads, d.headdim, d.dstate, d.rank
        G = groups(d)
        f32 = torch.float32
        shapes = dict(x=(Bsz, T, H, P, R), dt=(Bsz, T, H), lam=(Bsz, T, H),
                      A=(Bsz, T, H) if d.flags & M3_A_PER_TOKEN else (H,),
                      theta=(Bsz, T, G, N // 2), B=(Bsz, T, G, N, R), C=(Bsz, T, G, N, R),
                      h0=(Bsz, H, P, N), x_prev=(Bsz, H, P, R), B_prev=(Bsz, G, N, R))
        for k, t in (("x", x), ("dt", dt), ("lam", lam), ("theta", theta), ("B", B), ("C", C)):
            _check(k, t, shapes[k], ti)
        _check("A", A, shapes["A"], f32)
        _check("h0", h0, shapes["h0"], f32, optional=True)
        _check("x_prev", x_prev, shapes["x_prev"], ti, optional=True)
        _check("B_prev", B_prev, shapes["B_prev"], ti, optional=True)
        _check("dy", dy, shapes["x"], to)
        _check("dhT", dhT, shapes["h0"], f32, optional=True)
        for k in GRAD_NAMES:
            _check("d" + k, grads.get(k), shapes[k], f32,
                   optional=k in ("h0", "x_prev", "B_prev"))
    nbytes = 0
    if ws is not None:
        if not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous device tensor")
        nbytes = ws.numel() * ws.element_size()
    _check_bc(d)
    gp = lambda k: _ptr(grads.get(k))
    st = _lib().m3_scan_prefill_backward(
        ctypes.byref(d), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(theta), _ptr(B), _ptr(C),
        _ptr(h0), _ptr(x_prev), _ptr(B_prev), _ptr(dy), _ptr(dhT), gp("x"), gp("dt"), gp("A"),
        gp("lam"), gp("theta"), gp("B"), gp("C"), gp("h0"), gp("x_prev"), gp("B_prev"), _ptr(ws),
        nbytes, _stream(stream))
    if st != 0:
        raise M3Error(st, "m3_scan_prefill_backward")


def m3_prefill_varlen_workspace_size(dims: m3_dims) -> int:
    return int(_lib().m3_prefill_varlen_workspace_size(ctypes.byref(dims)))


def m3_scan_prefill_varlen(dims: m3_dims, cu_seqlens, x, dt, A, lam, theta, B, C, h0, x_prev,
                           B_prev, y, hT, ws, stream=None) -> None:
    """Packed sequences: dims.batch = S sequences, dims.seqlen = T total
    tokens; cu_seqlens is a device int32 tensor of S + 1 offsets."""
    d = dims
    ti, to = _TORCH.get(d.in_dtype), _TORCH.get(d.out_dtype)
    if ti is not None and to is not None:
        S, T, H, P, N, R = d.batch, d.seqlen, d.nheads, d.headdim, d.dstate, d.rank
        G = groups(d)
        _check("cu_seqlens", cu_seqlens, (S + 1,), torch.int32)
        _check("x", x, (T, H, P, R), ti)
        _check("dt", dt, (T, H), ti)
        _check("A", A, (T, H) if d.flags & M3_A_PER_TOKEN else (H,), torch.float32)
        _check("lam", lam, (T, H), ti)
        _check("theta", theta, (T, G, N // 2), ti, optional=_proj(d) is not None)
        if _proj(d) is not None:
            _proj(d).check((T,), G, N, ti)
        _check("B", B, (T, G, N, R), ti)
        _check("C", C, (T, G, N, R), ti)
        _check("h0", h0, (S, H, P, N), torch.float32, optional=True)
        _check("x_prev", x_prev, (S, H, P, R), ti, optional=True)
        _check("B_prev", B_prev, (S, G, N, R), ti, optional=True)
        _check("y", y, (T, H, P, R), to)
        _check("hT", hT, (S, H, P, N), torch.float32, optional=True)
    nbytes = 0
    if ws is not None:
        if not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous device tensor")
        nbytes = ws.numel() * ws.element_size()
    _check_bc(d)
    st = _lib().m3_scan_prefill_varlen(ctypes.byref(d), _ptr(cu_seqlens), _ptr(x), _ptr(dt),
                                       _ptr(A), _ptr(lam), _ptr(theta), _ptr(B), _ptr(C),
                                       _ptr(h0), _ptr(x_prev), _ptr(B_prev), _ptr(y), _ptr(hT),
                                       _ptr(ws), nbytes, _stream(stream))
    if st != 0:
        raise M3Error(st, "m3_scan_prefill_varlen")


def m3_decode_step(dims: m3_dims, h, x_t, x_prev, B_t, B_prev, C_t, dt_t, A, lam_t,
                   theta_t, y_t, stream=None) -> None:
    d = dims
    ti, to = _TORCH.get(d.in_dtype), _TORCH.get(d.out_dtype)
    if ti is not None and to is not None:
        Bsz, H, P, N, R = d.batch, d.nheads, d.headdim, d.dstate, d.rank
        G = groups(d)
        _check("h", h, (Bsz, H, P, N), torch.float32)
        _check("x_t", x_t, (Bsz, H, P, R), ti)
        _check("x_prev", x_prev, (Bsz, H, P, R), ti, optional=True)
        _check("B_t", B_t, (Bsz, G, N, R), ti)
        _check("B_prev", B_prev, (Bsz, G, N, R), ti, optional=True)
        _check("C_t", C_t, (Bsz, G, N, R), ti)
        _check("dt_t", dt_t, (Bsz, H), ti)
        _check("A", A, (Bsz, H) if d.flags & M3_A_PER_TOKEN else (H,), torch.float32)
        _check("lam_t", lam_t, (Bsz, H), ti)
        _check("theta_t", theta_t, (Bsz, G, N // 2), ti, optional=_proj(d) is not None)
        if _proj(d) is not None:
            _proj(d).check((Bsz,), G, N, ti)
        _check("y_t", y_t, (Bsz, H, P, R), to)
    _check_bc(d)
    st = _lib().m3_decode_step(ctypes.byref(d), _ptr(h), _ptr(x_t), _ptr(x_prev), _ptr(B_t),
                               _ptr(B_prev), _ptr(C_t), _ptr(dt_t), _ptr(A), _ptr(lam_t),
                               _ptr(theta_t), _ptr(y_t), _stream(stream))
    if st != 0:
        raise M3Error(st, "m3_decode_step")


def m3_decode_tokens(dims: m3_dims, h, x, x_prev, B, B_prev, C, dt, A, lam, theta, y,
                     stream=None) -> None:
    d = dims
    ti, to = _TORCH.get(d.in_dtype), _TORCH.get(d.out_dtype)
    if ti is not None and to is not None:
        Bsz, K, H, P, N, R = d.batch, d.seqlen, d.nheads, d.headdim, d.dstate, d.rank
        G = groups(d)
        _check("h", h, (Bsz, H, P, N), torch.float32)
        _check("x", x, (Bsz, K, H, P, R), ti)
        _check("x_prev", x_prev, (Bsz, H, P, R), ti, optional=True)
        _check("B", B, (Bsz, K, G, N, R), ti)
        _check("B_prev", B_prev, (Bsz, G, N, R), ti, optional=True)
        _check("C", C, (Bsz, K, G, N, R), ti)
        _check("dt", dt, (Bsz, K, H), ti)
        _check("A", A, (Bsz, K, H) if d.flags & M3_A_PER_TOKEN else (H,), torch.float32)
        _check("lam", lam, (Bsz, K, H), ti)
        _check("theta", theta, (Bsz, K, G, N // 2), ti)
        _check("y", y, (Bsz, K, H, P, R), to)
    _check_bc(d)
    st = _lib().m3_decode_tokens(ctypes.byref(d), _ptr(h), _ptr(x), _ptr(x_prev), _ptr(B),
                                 _ptr(B_prev), _ptr(C), _ptr(dt), _ptr(A), _ptr(lam),
                                 _ptr(theta), _ptr(y), _stream(stream))
    if st != 0:
        raise M3Error(st, "m3_decode_tokens")


# ---------------------------------------------------------------------------
# allocation helpers (torch only provides the memory)
def scan_prefill(x, dt, A, lam, theta, B, C, h0=None, x_prev=None, B_prev=None,
                 chunk=0, out_dtype=torch.float32, flags=0, want_hT=True, ws=None,
                 stream=None, bc=None, tp=None):
    """Allocate y (and hT, workspace) and call m3_scan_prefill.  Returns (y, hT).
    B, C and theta may have fewer head slots than x (head groups); with tp
    (a ThetaProj) theta may be None."""
    Bsz, T, H, P, R = x.shape
    G, N = B.shape[2], B.shape[3]
    d = make_dims(Bsz, T, H, P, N, R, chunk, dtype_code(x.dtype), dtype_code(out_dtype), flags,
                  0 if G == H else G, bc, tp)
    y = torch.empty((Bsz, T, H, P, R), dtype=out_dtype, device=x.device)
    hT = torch.empty((Bsz, H, P, N), dtype=torch.float32, device=x.device) if want_hT else None
    if ws is None:
        ws = workspace(d, x.device)
    m3_scan_prefill(d, x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, y, hT, ws, stream)
    return y, hT


def workspace(dims: m3_dims, device, varlen=False) -> torch.Tensor:
    n = (m3_prefill_varlen_workspace_size if varlen else m3_prefill_workspace_size)(dims)
    if n == 0:
        raise M3Error(2, "m3_prefill_workspace_size")
    return torch.empty((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def scan_prefill_backward(x, dt, A, lam, theta, B, C, dy, h0=None, x_prev=None, B_prev=None,
                          dhT=None, flags=0, chunk=0, stream=None) -> dict:
    """Allocate the fp32 gradients (and workspace) and call
    m3_scan_prefill_backward.  Returns a dict keyed by GRAD_NAMES."""
    Bsz, T, H, P, R = x.shape
    G, N = B.shape[2], B.shape[3]
    d = make_dims(Bsz, T, H, P, N, R, chunk, dtype_code(x.dtype), dtype_code(dy.dtype), flags,
                  0 if G == H else G)
    dev, f32 = x.device, torch.float32
    like = lambda t: None if t is None else torch.empty(t.shape, dtype=f32, device=dev)
    grads = {k: like(v) for k, v in (("x", x), ("dt", dt), ("A", A), ("lam", lam),
                                      ("theta", theta), ("B", B), ("C", C), ("x_prev", x_prev),
                                      ("B_prev", B_prev))}
    grads["h0"] = torch.empty((Bsz, H, P, N), dtype=f32, device=dev) if h0 is not None else None
    n = m3_prefill_backward_workspace_size(d)
    if n == 0:
        raise M3Error(2, "m3_prefill_backward_workspace_size")
    ws = torch.empty((n + 15) // 16 * 16, dtype=torch.uint8, device=dev)
    m3_scan_prefill_backward(d, x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, dy, dhT, grads,
                             ws, stream)
    return grads


def scan_prefill_varlen(cu_seqlens, x, dt, A, lam, theta, B, C, h0=None, x_prev=None,
                        B_prev=None, chunk=0, out_dtype=torch.float32, flags=0, want_hT=True,
                        ws=None, stream=None, bc=None, tp=None):
    """Allocate y (and hT, workspace) and call m3_scan_prefill_varlen on
    sequences packed into x [T, H, P, R].  Returns (y, hT)."""
    T, H, P, R = x.shape
    G, N = B.shape[1], B.shape[2]
    S = cu_seqlens.numel() - 1
    d = make_dims(S, T, H, P, N, R, chunk, dtype_code(x.dtype), dtype_code(out_dtype), flags,
                  0 if G == H else G, bc, tp)
    y = torch.empty((T, H, P, R), dtype=out_dtype, device=x.device)
    hT = torch.empty((S, H, P, N), dtype=torch.float32, device=x.device) if want_hT else None
    if ws is None:
        ws = workspace(d, x.device, varlen=True)
    m3_scan_prefill_varlen(d, cu_seqlens, x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, y,
                           hT, ws, stream)
    return y, hT


def decode_step(h, x_t, B_t, C_t, dt_t, A, lam_t, theta_t, x_prev=None, B_prev=None,
                out_dtype=torch.float32, flags=0, y_t=None, stream=None, bc=None, tp=None):
    """Advance h in place by one token; returns y_t (allocated unless given).
    B_t, C_t and theta_t may have fewer head slots than h (head groups);
    with tp (a ThetaProj) theta_t may be None."""
    Bsz, H, P, N = h.shape
    R = x_t.shape[-1]
    G = B_t.shape[1]
    d = make_dims(Bsz, 1, H, P, N, R, 0, dtype_code(x_t.dtype), dtype_code(out_dtype), flags,
                  0 if G == H else G, bc, tp)
    if y_t is None:
        y_t = torch.empty((Bsz, H, P, R), dtype=out_dtype, device=h.device)
    m3_decode_step(d, h, x_t, x_prev, B_t, B_prev, C_t, dt_t, A, lam_t, theta_t, y_t, stream)
    return y_t


def decode_tokens(h, x, B, C, dt, A, lam, theta, x_prev=None, B_prev=None,
                  out_dtype=torch.float32, flags=0, y=None, stream=None, bc=None):
    """Advance h in place by the K tokens of x ([Bsz, K, H, P, R]); returns y
    ([Bsz, K, H, P, R], allocated unless given)."""
    Bsz, K, H, P, R = x.shape
    N = h.shape[3]
    G = B.shape[2]
    d = make_dims(Bsz, K, H, P, N, R, 0, dtype_code(x.dtype), dtype_code(out_dtype), flags,
                  0 if G == H else G, bc)
    if y is None:
        y = torch.empty((Bsz, K, H, P, R), dtype=out_dtype, device=h.device)
    m3_decode_tokens(d, h, x, x_prev, B, B_prev, C, dt, A, lam, theta, y, stream)
    return y


# ---------------------------------------------------------------------------
# the other layers of a hybrid stack: gated recurrence, q/k norms with rotary
# positions, causal attention, gated delta rule, norms around a block
class _Switch:
    """The device of a call's tensors as the current one and, if given, the
    stream as the current one, so that what a helper allocates belongs to the
    stream that uses it."""

    def __init__(self, index, stream):
        self.device = torch.cuda.device(index)
        self.stream = torch.cuda.stream(stream)   # None: no change

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *e):
        self.stream.__exit__(*e)
        self.device.__exit__(*e)


_HERE = contextlib.nullcontext()


def _on(index, stream):
    """A context for the launch.  Nothing is switched where nothing has to be:
    a small call is bound by the host.  The launch goes to the tensors' device,
    so a stream of another one is refused."""
    if stream is None:
        if index == torch.cuda.current_device():
            return _HERE
    elif stream.device.index != index:
        raise ValueError(f"stream is of {stream.device}, the tensors are on cuda:{index}")
    return _Switch(index, stream)


def _raw(index):
    """The current stream of a device as the library takes it."""
    return torch._C._cuda_getCurrentRawStream(index)


def _same_device(names, *tensors):
    """All given tensors on one GPU; returns its index."""
    index = None
    for t in tensors:
        if t is not None:
            k = t.get_device() if isinstance(t, torch.Tensor) else -1
            if k != index:
                if index is not None or k < 0:
                    _device_error(names, tensors)
                index = k
    return index


def _device_error(names, tensors):
    for n, t in zip(names.split(), tensors):
        if t is not None and not (isinstance(t, torch.Tensor) and t.is_cuda):
            raise ValueError(f"{n} must be a device tensor")
    on = {n: str(t.device) for n, t in zip(names.split(), tensors) if t is not None}
    raise ValueError(f"tensors on several devices: {on}")


@functools.lru_cache(maxsize=256)
def _dims(kind, *fields):
    """The dims of a call, read only, with the reference that ctypes passes:
    equal calls share them."""
    d = kind(*fields)
    for (name, _), v in zip(kind._fields_, fields):   # ctypes cuts silently
        if isinstance(v, int) and getattr(d, name) != v:
            raise ValueError(f"{name}: {v} is out of range")
    return d, ctypes.byref(d)


def _addr(t):
    """A tensor's address as ctypes takes it for a void pointer."""
    return None if t is None else t.data_ptr()


def _dense(name, t, shape, dtype, optional=False):
    """_check for a tensor whose device is known."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(name, t, shape, dtype) -> int:
    """Checks a tensor of token rows that may be cut out of wider rows: the
    trailing (per-token) axes dense, consecutive tokens one stride apart
    across all leading axes.  Returns that stride, 0 for a dense tensor."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != expected {dtype}")
    if t.is_contiguous():
        return 0
    lead = 2 if len(shape) == 3 and name in _BATCHED else 1
    width = 1
    for n, st in zip(reversed(shape[lead:]), reversed(t.stride()[lead:])):
        if n != 1 and st != width:
            raise ValueError(f"{name}: a token's values must be contiguous")
        width *= n
    ld = t.stride(lead - 1) if shape[lead - 1] > 1 else max(t.stride(lead - 1), width)
    if shape[lead - 1] == 1 and lead == 2 and shape[0] > 1:
        ld = t.stride(0)
    if lead == 2 and shape[0] > 1 and shape[1] > 1 and t.stride(0) != shape[1] * ld:
        raise ValueError(f"{name}: sequences must follow each other without a gap")
    if ld < width:
        raise ValueError(f"{name}: token rows overlap")
    return ld


_BATCHED = ("x", "r", "i")


def _gated_setup(x, r, i, decay, c, cu_seqlens):
    packed = cu_seqlens is not None
    if x.dim() != (2 if packed else 3):
        raise ValueError("x must be [T, D] with cu_seqlens and [Bsz, T, D] without")
    D, dt = x.shape[-1], x.dtype
    code = dtype_code(dt)
    if packed:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must hold S + 1 offsets")
        B, T = cu_seqlens.numel() - 1, x.shape[0]
        _dense("cu_seqlens", cu_seqlens, (B + 1,), torch.int32)
    else:
        B, T = x.shape[:2]
    sh = x.shape
    _dense("decay", decay, (D,), torch.float32)
    d, ref = _dims(m3_gated_dims, B, T, D, code, c, _rows("x", x, sh, dt), _rows("r", r, sh, dt),
                   _rows("i", i, sh, dt), 0)
    return d, ref, packed


def _nst(T):
    return (T + M3_GATED_CHUNK - 1) // M3_GATED_CHUNK


def _ws(n, what, like):
    if n == 0:
        raise M3Error(2, what)
    return like.new_empty(((n + 15) // 16 * 16,), dtype=torch.uint8)


def gated_scan(x, r, i, decay, h0=None, c=8.0, cu_seqlens=None, want_hT=True, want_states=False,
               stream=None):
    """The gated linear recurrence over x, r, i [Bsz, T, D], or packed [T, D]
    with cu_seqlens (m3_gated_scan).  Returns (y, hT, states); states are for
    gated_scan_backward."""
    dev = _same_device("x r i decay h0 cu_seqlens", x, r, i, decay, h0, cu_seqlens)
    d, ref, packed = _gated_setup(x, r, i, decay, c, cu_seqlens)
    B, T, D = d.batch, d.seqlen, d.width
    _dense("h0", h0, (B, D), torch.float32, optional=True)
    lib = _lib()
    with _on(dev, stream):
        y = x.new_empty(x.shape)
        hT = decay.new_empty((B, D)) if want_hT else None
        st = None
        if want_states:
            st = decay.new_empty(((_nst(T),) if packed else (B, _nst(T))) + (D,))
        ws = _ws(lib.m3_gated_scan_workspace_size(ref, packed), "m3_gated_scan", x)
        e = lib.m3_gated_scan(ref, _addr(cu_seqlens), _addr(x), _addr(r), _addr(i),
                              _addr(decay), _addr(h0), _addr(y), _addr(hT), _addr(st), _addr(ws),
                              ws.numel(), _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_gated_scan")
    return y, hT, st


def gated_scan_backward(x, r, i, decay, dy, states, h0=None, dhT=None, c=8.0, cu_seqlens=None,
                        stream=None) -> dict:
    """Gradients of gated_scan (m3_gated_scan_backward): a dict with x, r, i
    in their dtype, decay and (if h0 is given) h0 in fp32.  Rows that no
    sequence covers are not written."""
    dev = _same_device("x r i decay dy states h0 dhT cu_seqlens", x, r, i, decay, dy, states, h0,
                       dhT, cu_seqlens)
    d, ref, packed = _gated_setup(x, r, i, decay, c, cu_seqlens)
    B, T, D = d.batch, d.seqlen, d.width
    _dense("h0", h0, (B, D), torch.float32, optional=True)
    _dense("dhT", dhT, (B, D), torch.float32, optional=True)
    _dense("dy", dy, x.shape, x.dtype)
    _dense("states", states, ((_nst(T),) if packed else (B, _nst(T))) + (D,), torch.float32)
    lib = _lib()
    with _on(dev, stream):
        g = {k: x.new_empty(x.shape) for k in ("x", "r", "i")}
        g["decay"] = decay.new_empty((D,))
        g["h0"] = decay.new_empty((B, D)) if h0 is not None else None
        ws = _ws(lib.m3_gated_scan_backward_workspace_size(ref, packed),
                 "m3_gated_scan_backward", x)
        e = lib.m3_gated_scan_backward(
            ref, _addr(cu_seqlens), _addr(x), _addr(r), _addr(i), _addr(decay), _addr(h0),
            _addr(states), _addr(dy), _addr(dhT), _addr(g["x"]), _addr(g["r"]), _addr(g["i"]),
            _addr(g["decay"]), _addr(g["h0"]), _addr(ws), ws.numel(), _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_gated_scan_backward")
    return g


def gated_step(h, x, r, i, decay, c=8.0, y=None, stream=None):
    """Advances h [Bsz, D] (fp32, in place) by one token of x, r, i [Bsz, D];
    returns y (allocated unless given)."""
    dev = _same_device("h x r i decay y", h, x, r, i, decay, y)
    if h.dim() != 2:
        raise ValueError("h must be [Bsz, D]")
    B, D = h.shape
    _dense("h", h, (B, D), torch.float32)
    _dense("decay", decay, (D,), torch.float32)
    dt, sh = x.dtype, h.shape
    _, ref = _dims(m3_gated_dims, B, 1, D, dtype_code(dt), c, _rows("x", x, sh, dt),
                   _rows("r", r, sh, dt), _rows("i", i, sh, dt), 0)
    with _on(dev, stream):
        if y is None:
            y = x.new_empty((B, D))
        else:
            _dense("y", y, sh, dt)
        e = _lib().m3_gated_step(ref, _addr(h), _addr(x), _addr(r), _addr(i),
                                 _addr(decay), _addr(y), _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_gated_step")
    return y


def _qk_setup(q, k, positions, q_weight, k_weight, eps, base, rotary_dim, flags):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [T, heads, headdim]")
    T, Hq, D = q.shape
    Hk = k.shape[1]
    code = dtype_code(q.dtype)
    ldq = _rows("q", q, (T, Hq, D), q.dtype)
    ldk = _rows("k", k, (T, Hk, D), q.dtype)
    _dense("positions", positions, (T,), torch.int32)
    _dense("q_weight", q_weight, (D,), torch.float32, optional=True)
    _dense("k_weight", k_weight, (D,), torch.float32, optional=True)
    return _dims(m3_qk_dims, T, Hq, Hk, D, D if rotary_dim is None else rotary_dim, code, flags,
                 eps, base, ldq, ldk, 0, 0)[1]


def qk_norm_rope(q, k, positions, q_weight=None, k_weight=None, eps=1e-6, base=10000.0,
                 rotary_dim=None, flags=0, stream=None):
    """RMS norms of q [T, Hq, D] and k [T, Hk, D] per head and their rotation
    by position (m3_qk_norm_rope).  Returns (q_out, k_out)."""
    dev = _same_device("q k positions q_weight k_weight", q, k, positions, q_weight, k_weight)
    ref = _qk_setup(q, k, positions, q_weight, k_weight, eps, base, rotary_dim, flags)
    with _on(dev, stream):
        qo, ko = q.new_empty(q.shape), k.new_empty(k.shape)
        e = _lib().m3_qk_norm_rope(ref, _addr(q), _addr(k), _addr(q_weight),
                                   _addr(k_weight), _addr(positions), _addr(qo), _addr(ko),
                                   _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_qk_norm_rope")
    return qo, ko


def qk_norm_rope_backward(q, k, positions, dq_out, dk_out, q_weight=None, k_weight=None, eps=1e-6,
                          base=10000.0, rotary_dim=None, flags=0, stream=None) -> dict:
    """Gradients of qk_norm_rope: a dict with q, k in their dtype and, for the
    weights that are given, q_weight, k_weight in fp32."""
    dev = _same_device("q k positions q_weight k_weight dq_out dk_out", q, k, positions, q_weight,
                       k_weight, dq_out, dk_out)
    ref = _qk_setup(q, k, positions, q_weight, k_weight, eps, base, rotary_dim, flags)
    _dense("dq_out", dq_out, q.shape, q.dtype)
    _dense("dk_out", dk_out, k.shape, q.dtype)
    lib = _lib()
    with _on(dev, stream):
        g = dict(q=q.new_empty(q.shape), k=q.new_empty(k.shape))
        for n, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            g[n] = None if w is None else w.new_empty(w.shape)
        ws = _ws(lib.m3_qk_norm_rope_backward_workspace_size(ref),
                 "m3_qk_norm_rope_backward", q)
        e = lib.m3_qk_norm_rope_backward(
            ref, _addr(q), _addr(k), _addr(q_weight), _addr(k_weight), _addr(positions),
            _addr(dq_out), _addr(dk_out), _addr(g["q"]), _addr(g["k"]), _addr(g["q_weight"]),
            _addr(g["k_weight"]), _addr(ws), ws.numel(), _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_qk_norm_rope_backward")
    return g


def _attn_setup(q, k, v, cu_q, cu_k, scale, ld_o=0, ld_do=0):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be [T, heads, headdim]")
    Tq, Hq, D = q.shape
    Tk, Hk = k.shape[:2]
    code = dtype_code(q.dtype)
    ld = [_rows("q", q, (Tq, Hq, D), q.dtype), _rows("k", k, (Tk, Hk, D), q.dtype),
          _rows("v", v, (Tk, Hk, D), q.dtype)]
    if cu_q.dim() != 1 or cu_q.numel() < 2:
        raise ValueError("cu_seqlens_q must hold S + 1 offsets")
    S = cu_q.numel() - 1
    _dense("cu_seqlens_q", cu_q, (S + 1,), torch.int32)
    _dense("cu_seqlens_k", cu_k, (S + 1,), torch.int32)
    return _dims(m3_attn_dims, S, Tq, Tk, Hq, Hk, D, code, D ** -0.5 if scale is None else scale,
                 *ld, ld_o, ld_do, 0, 0)[1]


def _split_ws(n, like):
    """The workspace of a call that may be split, and its bytes; none for the
    16 bytes that stand for a call that is not."""
    if n <= 16:
        return None, 0
    return like.new_empty(((n + 15) // 16 * 16,), dtype=torch.uint8), n


def attn_prefill_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, scale=None, stream=None):
    """Causal attention of packed sequences: q [Tq, Hq, D], k and v
    [Tk, Hk, D] (m3_attn_prefill_varlen; scale D^-1/2 by default).  Returns
    (o, lse).  Rows behind the last sequence are not written."""
    dev = _same_device("q k v cu_seqlens_q cu_seqlens_k", q, k, v, cu_seqlens_q, cu_seqlens_k)
    ref = _attn_setup(q, k, v, cu_seqlens_q, cu_seqlens_k, scale)
    lib = _lib()
    with _on(dev, stream):
        o = q.new_empty(q.shape)
        lse = q.new_empty(q.shape[:2], dtype=torch.float32)
        ws, n = _split_ws(lib.m3_attn_prefill_varlen_workspace_size(ref), q)
        e = lib.m3_attn_prefill_varlen(ref, _addr(cu_seqlens_q), _addr(cu_seqlens_k), _addr(q),
                                       _addr(k), _addr(v), _addr(o), _addr(lse), _addr(ws), n,
                                       _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_attn_prefill_varlen")
    return o, lse


def attn_prefill_varlen_backward(q, k, v, o, lse, d_o, cu_seqlens_q, cu_seqlens_k, scale=None,
                                 stream=None):
    """Gradients of attn_prefill_varlen for d_o: (dq, dk, dv)."""
    dev = _same_device("q k v o lse d_o cu_seqlens_q cu_seqlens_k", q, k, v, o, lse, d_o,
                       cu_seqlens_q, cu_seqlens_k)
    ref = _attn_setup(q, k, v, cu_seqlens_q, cu_seqlens_k, scale, _rows("o", o, q.shape, q.dtype),
                      _rows("d_o", d_o, q.shape, q.dtype))
    _dense("lse", lse, q.shape[:2], torch.float32)
    lib = _lib()
    with _on(dev, stream):
        dq, dk, dv = (q.new_empty(t.shape) for t in (q, k, v))
        ws = _ws(lib.m3_attn_prefill_varlen_backward_workspace_size(ref),
                 "m3_attn_prefill_varlen_backward", q)
        e = lib.m3_attn_prefill_varlen_backward(
            ref, _addr(cu_seqlens_q), _addr(cu_seqlens_k), _addr(q), _addr(k), _addr(v),
            _addr(o), _addr(lse), _addr(d_o), _addr(dq), _addr(dk), _addr(dv), _addr(ws), ws.numel(),
            _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_attn_prefill_varlen_backward")
    return dq, dk, dv


def attn_decode(q, k_cache, v_cache, lengths, scale=None, o=None, ws=None, stream=None):
    """One token per sequence, q [S, Hq, D], against caches [S, cap, Hk, D]
    holding lengths[s] rows (m3_attn_decode).  Returns (o, lse)."""
    dev = _same_device("q k_cache v_cache lengths o ws", q, k_cache, v_cache, lengths, o, ws)
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [S, Hq, D], the caches [S, cap, Hk, D]")
    S, Hq, D = q.shape
    if S == 0:
        raise ValueError("q holds no sequence")
    cap, Hk = k_cache.shape[1:3]
    code = dtype_code(q.dtype)
    strides = []
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if tuple(t.shape) != (S, cap, Hk, D):
            raise ValueError(f"{n}: shape {tuple(t.shape)} != expected {(S, cap, Hk, D)}")
        if S > 1 and (t.stride(0) <= 0):
            raise ValueError(f"{n}: sequences must not share rows")
        strides.append((_rows(n, t[0], (cap, Hk, D), q.dtype), t.stride(0) if S > 1 else 0))
    _dense("lengths", lengths, (S,), torch.int32)
    _, ref = _dims(m3_attn_dims, S, 0, cap, Hq, Hk, D, code, D ** -0.5 if scale is None else scale,
                   _rows("q", q, (S, Hq, D), q.dtype), strides[0][0], strides[1][0],
                   0 if o is None else _rows("o", o, q.shape, q.dtype), 0, strides[0][1],
                   strides[1][1])
    lib = _lib()
    with _on(dev, stream):
        if o is None:
            o = q.new_empty(q.shape)
        lse = q.new_empty((S, Hq), dtype=torch.float32)
        if ws is None:
            ws, n = _split_ws(lib.m3_attn_decode_workspace_size(ref), q)
        else:
            n = ws.numel() * ws.element_size()
        e = lib.m3_attn_decode(ref, _addr(lengths), _addr(q), _addr(k_cache),
                               _addr(v_cache), _addr(o), _addr(lse), _addr(ws), n, _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_attn_decode")
    return o, lse


def _flat(name, t, dims):
    """A dense call's [Bsz, T, ...] as token rows."""
    if t is None or t.dim() != dims:
        raise ValueError(f"{name} must have {dims} axes")
    try:
        return t.view(t.shape[0] * t.shape[1], *t.shape[2:])
    except RuntimeError:
        raise ValueError(f"{name}: sequences must follow each other without a gap") from None


def _delta_setup(q, k, v, g, beta, scale, cu_seqlens):
    """(dims, reference, packed, slots of chunks)"""
    packed = cu_seqlens is not None
    if packed:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must hold S + 1 offsets")
        if q.dim() != 3 or v.dim() != 3:
            raise ValueError("q, k and v must be [T, heads, headdim] with cu_seqlens")
        B, T = cu_seqlens.numel() - 1, q.shape[0]
        _dense("cu_seqlens", cu_seqlens, (B + 1,), torch.int32)
        rows, slots = T, T // M3_DELTA_CHUNK + B
    else:
        if q.dim() != 4:
            raise ValueError("q, k and v must be [Bsz, T, heads, headdim] without cu_seqlens")
        B, T = q.shape[:2]
        q, k, v = (_flat(n, t, 4) for n, t in (("q", q), ("k", k), ("v", v)))
        g, beta = (_flat(n, t, 3) for n, t in (("g", g), ("beta", beta)))
        rows, slots = B * T, B * ((T + M3_DELTA_CHUNK - 1) // M3_DELTA_CHUNK)
    Hk, Dk = q.shape[1:]
    Hv, Dv = v.shape[1:]
    dt = q.dtype
    d, ref = _dims(m3_delta_dims, B, T, Hk, Hv, Dk, Dv, dtype_code(dt),
                   Dk ** -0.5 if scale is None else scale, _rows("q", q, (rows, Hk, Dk), dt),
                   _rows("k", k, (rows, Hk, Dk), dt), _rows("v", v, (rows, Hv, Dv), dt),
                   _rows("g", g, (rows, Hv), dt), _rows("beta", beta, (rows, Hv), dt))
    return d, ref, packed, slots


def m3_delta_state_floats(dk, dv):
    """M3_DELTA_STATE_FLOATS: what delta_scan saves of a chunk and head."""
    return (dk + 64) * dv + 64 * 64 + 5 * 64


def _delta_states(d, slots):
    return (slots, d.nheads_v, m3_delta_state_floats(d.headdim_k, d.headdim_v))


def delta_scan(q, k, v, g, beta, h0=None, scale=None, cu_seqlens=None, want_hT=True,
               want_states=False, stream=None):
    """The gated delta rule over q, k [Bsz, T, Hk, Dk], v [Bsz, T, Hv, Dv], g
    and beta [Bsz, T, Hv], or packed without Bsz and with cu_seqlens
    (m3_delta_scan; scale Dk^-1/2 by default).  Returns (o, hT, states);
    states are for delta_scan_backward."""
    dev = _same_device("q k v g beta h0 cu_seqlens", q, k, v, g, beta, h0, cu_seqlens)
    d, ref, packed, slots = _delta_setup(q, k, v, g, beta, scale, cu_seqlens)
    state = (d.batch, d.nheads_v, d.headdim_k, d.headdim_v)
    _dense("h0", h0, state, torch.float32, optional=True)
    lib = _lib()
    with _on(dev, stream):
        o = v.new_empty(v.shape)
        hT = v.new_empty(state, dtype=torch.float32) if want_hT else None
        st = None
        if want_states:
            st = v.new_empty(_delta_states(d, slots), dtype=torch.float32)
        ws = _ws(lib.m3_delta_scan_workspace_size(ref, packed), "m3_delta_scan", q)
        e = lib.m3_delta_scan(ref, _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(g),
                              _addr(beta), _addr(h0), _addr(o), _addr(hT), _addr(st), _addr(ws),
                              ws.numel(), _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_delta_scan")
    return o, hT, st


def delta_scan_backward(q, k, v, g, beta, d_o, states, h0=None, dhT=None, scale=None,
                        cu_seqlens=None, stream=None) -> dict:
    """Gradients of delta_scan (m3_delta_scan_backward): a dict with q, k, v,
    g, beta in their dtype and (if h0 is given) h0 in fp32.  Rows that no
    sequence covers are not written."""
    dev = _same_device("q k v g beta d_o states h0 dhT cu_seqlens", q, k, v, g, beta, d_o, states,
                       h0, dhT, cu_seqlens)
    d, ref, packed, slots = _delta_setup(q, k, v, g, beta, scale, cu_seqlens)
    state = (d.batch, d.nheads_v, d.headdim_k, d.headdim_v)
    _dense("h0", h0, state, torch.float32, optional=True)
    _dense("dhT", dhT, state, torch.float32, optional=True)
    _dense("d_o", d_o, v.shape, v.dtype)
    _dense("states", states, _delta_states(d, slots), torch.float32)
    lib = _lib()
    with _on(dev, stream):
        r = {n: t.new_empty(t.shape) for n, t in (("q", q), ("k", k), ("v", v), ("g", g),
                                                  ("beta", beta))}
        r["h0"] = None if h0 is None else h0.new_empty(state)
        ws = _ws(lib.m3_delta_scan_backward_workspace_size(ref, packed),
                 "m3_delta_scan_backward", q)
        e = lib.m3_delta_scan_backward(
            ref, _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(g), _addr(beta),
            _addr(states), _addr(d_o), _addr(dhT), _addr(r["q"]), _addr(r["k"]), _addr(r["v"]),
            _addr(r["g"]), _addr(r["beta"]), _addr(r["h0"]), _addr(ws), ws.numel(), _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_delta_scan_backward")
    return r


def delta_step(h, q, k, v, g, beta, scale=None, o=None, stream=None):
    """Advances h [Bsz, Hv, Dk, Dv] (fp32, in place) by one token of q, k
    [Bsz, Hk, Dk], v [Bsz, Hv, Dv], g and beta [Bsz, Hv]; returns o (allocated
    unless given)."""
    dev = _same_device("h q k v g beta o", h, q, k, v, g, beta, o)
    if h.dim() != 4 or q.dim() != 3:
        raise ValueError("h must be [Bsz, Hv, Dk, Dv], q and k [Bsz, Hk, Dk]")
    B, Hv, Dk, Dv = h.shape
    Hk, dt = q.shape[1], q.dtype
    _dense("h", h, h.shape, torch.float32)
    _, ref = _dims(m3_delta_dims, B, 1, Hk, Hv, Dk, Dv, dtype_code(dt),
                   Dk ** -0.5 if scale is None else scale, _rows("q", q, (B, Hk, Dk), dt),
                   _rows("k", k, (B, Hk, Dk), dt), _rows("v", v, (B, Hv, Dv), dt),
                   _rows("g", g, (B, Hv), dt), _rows("beta", beta, (B, Hv), dt))
    with _on(dev, stream):
        if o is None:
            o = v.new_empty(v.shape)
        else:
            _dense("o", o, v.shape, dt)
        e = _lib().m3_delta_step(ref, _addr(h), _addr(q), _addr(k), _addr(v), _addr(g),
                                 _addr(beta), _addr(o), _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_delta_step")
    return o


def _block_setup(x, y, gate, y_weight, scale, n_weight, eps, flags):
    if x.dim() != 2:
        raise ValueError("x must be [T, W]")
    T, W = x.shape
    code = dtype_code(x.dtype)
    lds = [_rows("x", x, x.shape, x.dtype), _rows("y", y, x.shape, x.dtype),
           0 if gate is None else _rows("gate", gate, x.shape, x.dtype)]
    for n, t in (("y_weight", y_weight), ("scale", scale), ("n_weight", n_weight)):
        _dense(n, t, (W,), torch.float32, optional=True)
    return _dims(m3_block_dims, T, W, code, flags, eps, *lds)[1]


def block_norm(x, y, gate=None, y_weight=None, scale=None, n_weight=None, eps=1e-6, flags=0,
               want_n=True, stream=None):
    """A block's output y [T, W] normed, gated, scaled and added to the
    residual stream x, and the stream normed for the next block
    (m3_block_norm).  Returns (h, n)."""
    dev = _same_device("x y gate y_weight scale n_weight", x, y, gate, y_weight, scale, n_weight)
    ref = _block_setup(x, y, gate, y_weight, scale, n_weight, eps, flags)
    with _on(dev, stream):
        h = x.new_empty(x.shape)
        n = x.new_empty(x.shape) if want_n else None
        e = _lib().m3_block_norm(ref, _addr(x), _addr(y), _addr(gate), _addr(y_weight),
                                 _addr(scale), _addr(n_weight), _addr(h), _addr(n), _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_block_norm")
    return h, n


def block_norm_backward(x, y, dh, dn, gate=None, y_weight=None, scale=None, n_weight=None,
                        eps=1e-6, flags=0, stream=None) -> dict:
    """Gradients of block_norm for dh and dn (one of them may be None): a dict
    with x, y and gate in their dtype and, for those that are given, y_weight,
    scale and n_weight in fp32."""
    dev = _same_device("x y dh dn gate y_weight scale n_weight", x, y, dh, dn, gate, y_weight,
                       scale, n_weight)
    ref = _block_setup(x, y, gate, y_weight, scale, n_weight, eps, flags)
    _dense("dh", dh, x.shape, x.dtype, optional=True)
    _dense("dn", dn, x.shape, x.dtype, optional=True)
    lib = _lib()
    with _on(dev, stream):
        g = {n: None if t is None else t.new_empty(t.shape) for n, t in
             (("x", x), ("y", y), ("gate", gate), ("y_weight", y_weight), ("scale", scale),
              ("n_weight", n_weight))}
        ws = _ws(lib.m3_block_norm_backward_workspace_size(ref), "m3_block_norm_backward", x)
        e = lib.m3_block_norm_backward(
            ref, _addr(x), _addr(y), _addr(gate), _addr(y_weight), _addr(scale), _addr(n_weight),
            _addr(dh), _addr(dn), _addr(g["x"]), _addr(g["y"]), _addr(g["gate"]),
            _addr(g["y_weight"]), _addr(g["scale"]), _addr(g["n_weight"]), _addr(ws), ws.numel(),
            _raw(dev))
    if e != 0:
        raise M3Error(e, "m3_block_norm_backward")
    return g
