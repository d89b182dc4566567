"""Thin ctypes binding of libgdn.so (C ABI in include/gdn.h).

Argument marshalling only: shape/dtype checks, device pointers, the current
torch stream, and workspace allocation through torch.  Every step of the
computation runs in the library's CUDA kernels.  Importing this module loads the
library and raises if it is missing -- there is no other implementation.
"""
from __future__ import annotations

import ctypes
import os
from itertools import accumulate

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
PATH_NONE, PATH_SIMT, PATH_TCGEN05 = 0, 1, 2
PATH_NAMES = {PATH_NONE: "none", PATH_SIMT: "simt", PATH_TCGEN05: "tcgen05"}


class GdnError(RuntimeError):
    pass


def library_path() -> str:
    return _LIB_PATH


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"libgdn.so not found at {_LIB_PATH}: build it with "
            "`python -m gated_delta_rule_130_b200.build` (there is no fallback path)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, fp, I, Z = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.gdn_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, I, I, I, I, I, I, I, vp, Z, vp]
    lib.gdn_chunk_fwd.restype = I
    lib.gdn_chunk_fwd_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.gdn_chunk_fwd_workspace_size.restype = Z
    lib.gdn_chunk_fwd_path.argtypes = [I, I, I, I, I, I, I]
    lib.gdn_chunk_fwd_path.restype = I
    lib.gdn_chunk_fwd_variant.argtypes = [I, I, I, I, I, I, I]
    lib.gdn_chunk_fwd_variant.restype = I
    lib.gdn_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, vp, I, I, I, I, I, vp]
    lib.gdn_decode_step.restype = I
    U = ctypes.c_uint
    lib.gdn_chunk_fwd_ex.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, I, I, I, I, I, I, I, U, vp,
                                     Z, vp]
    lib.gdn_chunk_fwd_ex.restype = I
    lib.gdn_chunk_fwd_workspace_size_ex.argtypes = [I, I, I, I, I, I, I, U]
    lib.gdn_chunk_fwd_workspace_size_ex.restype = Z
    lib.gdn_decode_step_ex.argtypes = [vp, vp, vp, fp, fp, fp, vp, I, I, I, I, I, U, vp]
    lib.gdn_decode_step_ex.restype = I
    lib.gdn_chunk_fwd_varlen.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, vp, vp, I, I, I, I, I, I,
                                         U, vp, Z, vp]
    lib.gdn_chunk_fwd_varlen.restype = I
    lib.gdn_chunk_fwd_varlen_workspace_size.argtypes = [vp, I, I, I, I, I, I, U]
    lib.gdn_chunk_fwd_varlen_workspace_size.restype = Z
    lib.gdn_chunk_bwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, vp, vp, vp, fp, fp, fp, I, I, I,
                                  I, I, I, I, vp, Z, vp]
    lib.gdn_chunk_bwd.restype = I
    lib.gdn_chunk_bwd_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.gdn_chunk_bwd_workspace_size.restype = Z
    lib.gdn_chunk_bwd_path.argtypes = [I, I, I, I, I, I, I]
    lib.gdn_chunk_bwd_path.restype = I
    lib.gdn_chunk_fwd_cw.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp, fp, I, I, I, I, I, I, I, vp,
                                     Z, vp]
    lib.gdn_chunk_fwd_cw.restype = I
    lib.gdn_chunk_fwd_cw_path.argtypes = [I, I, I, I, I, I, I]
    lib.gdn_chunk_fwd_cw_path.restype = I
    lib.gdn_chunk_fwd_cw_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.gdn_chunk_fwd_cw_workspace_size.restype = Z
    lib.gdn_decode_step_cw.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp, I, I, I, I, I, vp]
    lib.gdn_decode_step_cw.restype = I
    L, Fl = ctypes.c_longlong, ctypes.c_float
    lib.gdn_decode_runs.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, vp, I, I, I, I, I, I, I, L, L,
                                    L, L, L, I, U, vp]
    lib.gdn_decode_runs.restype = I
    lib.gdn_short_conv_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, L, I,
                                       I, I, vp]
    lib.gdn_short_conv_fwd.restype = I
    lib.gdn_short_conv_bwd.argtypes = [vp, vp, vp, I, vp, vp, vp, vp, vp, fp, fp, I, I, I, I, L, I,
                                       I, I, vp, Z, vp]
    lib.gdn_short_conv_bwd.restype = I
    lib.gdn_short_conv_bwd_workspace_size.argtypes = [I, I, I]
    lib.gdn_short_conv_bwd_workspace_size.restype = Z
    lib.gdn_rms_norm_fwd.argtypes = [vp, vp, vp, vp, vp, fp, vp, I, I, I, I, L, L, L, Fl, I, I, vp]
    lib.gdn_rms_norm_fwd.restype = I
    lib.gdn_rms_norm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, fp, vp, I, I, I, L, L, L, L, Fl, I, I,
                                     vp, Z, vp]
    lib.gdn_rms_norm_bwd.restype = I
    lib.gdn_rms_norm_bwd_workspace_size.argtypes = [I, I, I]
    lib.gdn_rms_norm_bwd_workspace_size.restype = Z
    lib.gdn_debug_withhold_first_arrival.argtypes = [I]
    lib.gdn_debug_withhold_first_arrival.restype = I
    lib.gdn_check_device_status.argtypes = []
    lib.gdn_check_device_status.restype = I
    lib.gdn_status_string.argtypes = [I]
    lib.gdn_status_string.restype = ctypes.c_char_p
    return lib


LIB = _load()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDN_F32
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    raise GdnError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _check(status: int, what: str):
    if status != 0:
        raise GdnError(f"{what}: {LIB.gdn_status_string(status).decode()} (status {status})")


def _dev(t: torch.Tensor, name: str, dtype=None, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GdnError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise GdnError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise GdnError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise GdnError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


def _stream_ptr(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def check_device_status():
    """Synchronise and raise if a fused tensor-core kernel timed out since the last check."""
    _check(int(LIB.gdn_check_device_status()), "gdn_check_device_status")


# Input prologue flags of the _ex entry points (gdn_flag_t in include/gdn.h).
GDN_FLAG_L2NORM_QK = 1
GDN_FLAG_GATE_LOGITS = 2


def _flags(l2norm_qk: bool, gate_logits: bool) -> int:
    return (GDN_FLAG_L2NORM_QK if l2norm_qk else 0) | (GDN_FLAG_GATE_LOGITS if gate_logits else 0)


def chunk_fwd_workspace_size(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16,
                             l2norm_qk: bool = False, gate_logits: bool = False) -> int:
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(LIB.gdn_chunk_fwd_workspace_size_ex(B, T, H, Dk, Dv, chunk, code,
                                                   _flags(l2norm_qk, gate_logits)))


def chunk_fwd_path(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16) -> str:
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    p = int(LIB.gdn_chunk_fwd_path(B, T, H, Dk, Dv, chunk, code))
    if p < 0:
        raise GdnError("invalid or unsupported sizes")
    return PATH_NAMES[p]


VARIANT_NAMES = {0: None, 1: "fused", 2: "precomputed", 3: "split"}


def chunk_fwd_variant(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16):
    """Which tcgen05 variant a chunk_fwd call with these sizes runs: "fused",
    "precomputed", or None off the tcgen05 path."""
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return VARIANT_NAMES[int(LIB.gdn_chunk_fwd_variant(B, T, H, Dk, Dv, chunk, code))]


def chunk_fwd(q, k, v, log_alpha, beta, S0=None, chunk: int = 64, out=None, S_T=None,
              return_state: bool = True, workspace=None, l2norm_qk: bool = False,
              gate_logits: bool = False):
    """Chunkwise forward: returns (o [B,T,H,Dv], S_T [B,H,Dv,Dk] float32 or None).

    q, k [B,T,H,Dk] and v [B,T,H,Dv] in float32 or bfloat16 (same type);
    log_alpha, beta [B,T,H] float32; S0 [B,H,Dv,Dk] float32 or None (zeros).
    ``S_T`` may be passed (and may be ``S0`` itself for in-place continuation).
    ``l2norm_qk``: q and k are raw and get normalised per token and head in the
    kernels; ``gate_logits``: log_alpha and beta hold logits (log alpha =
    -softplus(x), beta = sigmoid(y)).
    """
    flags = _flags(l2norm_qk, gate_logits)
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise GdnError("q, k must be [B,T,H,Dk] and v [B,T,H,Dv]")
    B, T, H, Dk = q.shape
    Dv = v.shape[3]
    dev = q.device
    code = _dtype_code(q)
    args = [_dev(q, "q", q.dtype, dev), _dev(k, "k", q.dtype, dev), _dev(v, "v", q.dtype, dev)]
    if log_alpha.shape != (B, T, H) or beta.shape != (B, T, H):
        raise GdnError("log_alpha and beta must be [B,T,H]")
    args += [_dev(log_alpha, "log_alpha", torch.float32, dev),
             _dev(beta, "beta", torch.float32, dev)]
    if S0 is not None:
        if S0.shape != (B, H, Dv, Dk):
            raise GdnError("S0 must be [B,H,Dv,Dk]")
        args.append(_dev(S0, "S0", torch.float32, dev))
    else:
        args.append(None)
    o = out if out is not None else torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
    if o.shape != (B, T, H, Dv):
        raise GdnError("out must be [B,T,H,Dv]")
    args.append(_dev(o, "out", q.dtype, dev))
    if S_T is None and return_state:
        S_T = torch.empty((B, H, Dv, Dk), dtype=torch.float32, device=dev)
    if S_T is not None:
        if S_T.shape != (B, H, Dv, Dk):
            raise GdnError("S_T must be [B,H,Dv,Dk]")
        args.append(_dev(S_T, "S_T", torch.float32, dev))
    else:
        args.append(None)
    need = int(LIB.gdn_chunk_fwd_workspace_size_ex(B, T, H, Dk, Dv, chunk, code, flags))
    ws_ptr, ws_bytes = None, 0
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    st = LIB.gdn_chunk_fwd_ex(*args, B, T, H, Dk, Dv, chunk, code, flags, ws_ptr, ws_bytes,
                              _stream_ptr(dev))
    _check(st, "gdn_chunk_fwd")
    return o, S_T


def chunk_bwd_workspace_size(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16) -> int:
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(LIB.gdn_chunk_bwd_workspace_size(B, T, H, Dk, Dv, chunk, code))


def chunk_bwd(q, k, v, log_alpha, beta, S0, d_o, dS_T=None, chunk: int = 64, workspace=None,
              want_dS0: bool = True):
    """Chunkwise backward of ``chunk_fwd`` (plain gates, no prologue).

    Given the forward's inputs and d_o = dL/do [B,T,H,Dv] (q's dtype), dS_T =
    dL/dS_T [B,H,Dv,Dk] float32 or None, returns (dq, dk, dv, dlog_alpha, dbeta,
    dS0): dq, dk, dv in q's dtype, the rest float32 (dS0 None unless want_dS0).
    """
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise GdnError("q, k must be [B,T,H,Dk] and v [B,T,H,Dv]")
    B, T, H, Dk = q.shape
    Dv = v.shape[3]
    dev = q.device
    code = _dtype_code(q)
    if log_alpha.shape != (B, T, H) or beta.shape != (B, T, H):
        raise GdnError("log_alpha and beta must be [B,T,H]")
    if d_o.shape != v.shape:
        raise GdnError("d_o must be [B,T,H,Dv]")
    state = (B, H, Dv, Dk)
    for x, n in ((S0, "S0"), (dS_T, "dS_T")):
        if x is not None and x.shape != state:
            raise GdnError(f"{n} must be [B,H,Dv,Dk]")
    opt = lambda x, n: _dev(x, n, torch.float32, dev) if x is not None else None
    args = [_dev(q, "q", q.dtype, dev), _dev(k, "k", q.dtype, dev), _dev(v, "v", q.dtype, dev),
            _dev(log_alpha, "log_alpha", torch.float32, dev),
            _dev(beta, "beta", torch.float32, dev), opt(S0, "S0"),
            _dev(d_o, "d_o", q.dtype, dev), opt(dS_T, "dS_T")]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dla = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    dbe = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    dS0 = torch.empty(state, dtype=torch.float32, device=dev) if want_dS0 else None
    args += [dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dla.data_ptr(), dbe.data_ptr(),
             dS0.data_ptr() if dS0 is not None else None]
    need = int(LIB.gdn_chunk_bwd_workspace_size(B, T, H, Dk, Dv, chunk, code))
    ws_ptr, ws_bytes = None, 0
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    st = LIB.gdn_chunk_bwd(*args, B, T, H, Dk, Dv, chunk, code, ws_ptr, ws_bytes,
                           _stream_ptr(dev))
    _check(st, "gdn_chunk_bwd")
    return dq, dk, dv, dla, dbe, dS0


def chunk_bwd_path(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16) -> str:
    """Which kernels chunk_bwd runs for these sizes: "tcgen05", "simt" or "none"."""
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    st = int(LIB.gdn_chunk_bwd_path(B, T, H, Dk, Dv, chunk, code))
    if st < 0:
        raise GdnError("gdn_chunk_bwd_path: invalid sizes")
    return PATH_NAMES[st]


def chunk_fwd_cw_path(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16) -> str:
    """Which kernels chunk_fwd_cw runs for these sizes: "tcgen05", "simt" or "none"."""
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    st = int(LIB.gdn_chunk_fwd_cw_path(B, T, H, Dk, Dv, chunk, code))
    if st < 0:
        raise GdnError("gdn_chunk_fwd_cw_path: invalid sizes")
    return PATH_NAMES[st]


def chunk_fwd_cw_workspace_size(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16) -> int:
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(LIB.gdn_chunk_fwd_cw_workspace_size(B, T, H, Dk, Dv, chunk, code))


def chunk_fwd_cw(q, k, v, log_alpha, b, w, S0=None, chunk: int = 64, out=None, S_T=None,
                 return_state: bool = True, workspace=None):
    """Channel-wise gates: S_t = S_{t-1} Diag(alpha_t)(I - (b_t o k_t) k_t^T) + (w_t o v_t) k_t^T.

    q, k [B,T,H,Dk], v [B,T,H,Dv] (float32 or bfloat16); log_alpha, b
    [B,T,H,Dk] and w [B,T,H,Dv] float32; S0 [B,H,Dv,Dk] float32 or None.
    Returns (o [B,T,H,Dv], S_T or None).
    """
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise GdnError("q, k must be [B,T,H,Dk] and v [B,T,H,Dv]")
    B, T, H, Dk = q.shape
    Dv = v.shape[3]
    dev = q.device
    code = _dtype_code(q)
    if log_alpha.shape != q.shape or b.shape != q.shape or w.shape != v.shape:
        raise GdnError("log_alpha and b must be [B,T,H,Dk] and w [B,T,H,Dv]")
    args = [_dev(q, "q", q.dtype, dev), _dev(k, "k", q.dtype, dev), _dev(v, "v", q.dtype, dev),
            _dev(log_alpha, "log_alpha", torch.float32, dev), _dev(b, "b", torch.float32, dev),
            _dev(w, "w", torch.float32, dev)]
    state = (B, H, Dv, Dk)
    if S0 is not None and S0.shape != state:
        raise GdnError("S0 must be [B,H,Dv,Dk]")
    args.append(_dev(S0, "S0", torch.float32, dev) if S0 is not None else None)
    o = out if out is not None else torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
    if o.shape != (B, T, H, Dv):
        raise GdnError("out must be [B,T,H,Dv]")
    args.append(_dev(o, "out", q.dtype, dev))
    if S_T is None and return_state:
        S_T = torch.empty(state, dtype=torch.float32, device=dev)
    if S_T is not None and S_T.shape != state:
        raise GdnError("S_T must be [B,H,Dv,Dk]")
    args.append(_dev(S_T, "S_T", torch.float32, dev) if S_T is not None else None)
    need = int(LIB.gdn_chunk_fwd_cw_workspace_size(B, T, H, Dk, Dv, chunk, code))
    ws_ptr, ws_bytes = None, 0
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    st = LIB.gdn_chunk_fwd_cw(*args, B, T, H, Dk, Dv, chunk, code, ws_ptr, ws_bytes,
                              _stream_ptr(dev))
    _check(st, "gdn_chunk_fwd_cw")
    return o, S_T


def decode_step_cw(q, k, v, log_alpha, b, w, S, out=None):
    """One channel-wise-gate step for every (b, h); S [B,H,Dv,Dk] updated in place.
    q, k, log_alpha, b [B,H,Dk]; v, w [B,H,Dv].  Returns o [B,H,Dv]."""
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise GdnError("q, k must be [B,H,Dk] and v [B,H,Dv]")
    B, H, Dk = q.shape
    Dv = v.shape[2]
    dev = q.device
    if log_alpha.shape != q.shape or b.shape != q.shape or w.shape != v.shape:
        raise GdnError("log_alpha and b must be [B,H,Dk] and w [B,H,Dv]")
    if S.shape != (B, H, Dv, Dk):
        raise GdnError("S must be [B,H,Dv,Dk]")
    o = out if out is not None else torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
    st = LIB.gdn_decode_step_cw(
        _dev(q, "q", q.dtype, dev), _dev(k, "k", q.dtype, dev), _dev(v, "v", q.dtype, dev),
        _dev(log_alpha, "log_alpha", torch.float32, dev), _dev(b, "b", torch.float32, dev),
        _dev(w, "w", torch.float32, dev), _dev(S, "S", torch.float32, dev),
        _dev(o, "out", q.dtype, dev), B, H, Dk, Dv, _dtype_code(q), _stream_ptr(dev))
    _check(st, "gdn_decode_step_cw")
    return o


def _host_offsets(cu_seqlens) -> torch.Tensor:
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int32).cpu().contiguous()
    if cu.dim() != 1 or cu.numel() < 1:
        raise GdnError("cu_seqlens must be a 1-D list of N + 1 offsets")
    return cu


def chunk_fwd_varlen_workspace_size(cu_seqlens, H, Dk, Dv, chunk=64, dtype=torch.bfloat16,
                                    l2norm_qk: bool = False, gate_logits: bool = False) -> int:
    cu = _host_offsets(cu_seqlens)
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(LIB.gdn_chunk_fwd_varlen_workspace_size(cu.data_ptr(), cu.numel() - 1, H, Dk, Dv,
                                                       chunk, code, _flags(l2norm_qk, gate_logits)))


def chunk_fwd_varlen(q, k, v, log_alpha, beta, cu_seqlens, S0=None, chunk: int = 64, out=None,
                     S_T=None, return_state: bool = True, workspace=None, l2norm_qk: bool = False,
                     gate_logits: bool = False, cu_seqlens_device=None):
    """Chunkwise forward over N variable-length sequences packed without padding.

    q, k [total, H, Dk], v [total, H, Dv], log_alpha, beta [total, H]; ``cu_seqlens``
    the N + 1 token offsets (host list or tensor; sequence n is tokens
    cu_seqlens[n] .. cu_seqlens[n + 1] - 1).  S0 / S_T are [N, H, Dv, Dk] float32.
    ``cu_seqlens_device``: the same offsets as an int32 tensor on q's device (else
    they are copied there on every call, a synchronous copy).
    Returns (o [total, H, Dv], S_T or None).
    """
    cu = _host_offsets(cu_seqlens)
    N = cu.numel() - 1
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise GdnError("q, k must be [total,H,Dk] and v [total,H,Dv]")
    total, H, Dk = q.shape
    Dv = v.shape[2]
    if int(cu[-1]) != total:
        raise GdnError("cu_seqlens[-1] must equal the number of packed tokens")
    dev = q.device
    code = _dtype_code(q)
    flags = _flags(l2norm_qk, gate_logits)
    if log_alpha.shape != (total, H) or beta.shape != (total, H):
        raise GdnError("log_alpha and beta must be [total,H]")
    args = [_dev(q, "q", q.dtype, dev), _dev(k, "k", q.dtype, dev), _dev(v, "v", q.dtype, dev),
            _dev(log_alpha, "log_alpha", torch.float32, dev), _dev(beta, "beta", torch.float32, dev)]
    if S0 is not None:
        if S0.shape != (N, H, Dv, Dk):
            raise GdnError("S0 must be [N,H,Dv,Dk]")
        args.append(_dev(S0, "S0", torch.float32, dev))
    else:
        args.append(None)
    o = out if out is not None else torch.empty((total, H, Dv), dtype=q.dtype, device=dev)
    if o.shape != (total, H, Dv):
        raise GdnError("out must be [total,H,Dv]")
    args.append(_dev(o, "out", q.dtype, dev))
    if S_T is None and return_state:
        S_T = torch.empty((N, H, Dv, Dk), dtype=torch.float32, device=dev)
    if S_T is not None:
        if S_T.shape != (N, H, Dv, Dk):
            raise GdnError("S_T must be [N,H,Dv,Dk]")
        args.append(_dev(S_T, "S_T", torch.float32, dev))
    else:
        args.append(None)
    if cu_seqlens_device is not None:
        if cu_seqlens_device.shape != cu.shape:
            raise GdnError("cu_seqlens_device must hold the N + 1 offsets")
        _dev(cu_seqlens_device, "cu_seqlens_device", torch.int32, dev)
        cu_dev = cu_seqlens_device
    else:
        cu_dev = cu.to(dev)
    need = int(LIB.gdn_chunk_fwd_varlen_workspace_size(cu.data_ptr(), N, H, Dk, Dv, chunk, code,
                                                       flags))
    ws_ptr, ws_bytes = None, 0
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    st = LIB.gdn_chunk_fwd_varlen(*args, cu_dev.data_ptr(), cu.data_ptr(), N, H, Dk, Dv, chunk,
                                  code, flags, ws_ptr, ws_bytes, _stream_ptr(dev))
    _check(st, "gdn_chunk_fwd_varlen")
    return o, S_T


def decode_step(q, k, v, log_alpha, beta, S, out=None, l2norm_qk: bool = False,
                gate_logits: bool = False):
    """One recurrent step for every (b,h); S [B,H,Dv,Dk] float32 is updated in place.

    q, k [B,H,Dk], v [B,H,Dv] float32 or bfloat16; log_alpha, beta [B,H] float32.
    Returns o [B,H,Dv] in q's dtype.  ``l2norm_qk`` / ``gate_logits``: the input
    prologue, as in ``chunk_fwd``.
    """
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise GdnError("q, k must be [B,H,Dk] and v [B,H,Dv]")
    B, H, Dk = q.shape
    Dv = v.shape[2]
    dev = q.device
    code = _dtype_code(q)
    if log_alpha.shape != (B, H) or beta.shape != (B, H) or S.shape != (B, H, Dv, Dk):
        raise GdnError("log_alpha, beta must be [B,H] and S [B,H,Dv,Dk]")
    o = out if out is not None else torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
    st = LIB.gdn_decode_step_ex(
        _dev(q, "q", q.dtype, dev), _dev(k, "k", q.dtype, dev), _dev(v, "v", q.dtype, dev),
        _dev(log_alpha, "log_alpha", torch.float32, dev), _dev(beta, "beta", torch.float32, dev),
        _dev(S, "S", torch.float32, dev), _dev(o, "out", q.dtype, dev), B, H, Dk, Dv, code,
        _flags(l2norm_qk, gate_logits), _stream_ptr(dev))
    _check(st, "gdn_decode_step")
    return o


# ---------------------------------------------------------------------------
# The operators around the rule (gdn_decode_runs, gdn_short_conv_*, gdn_rms_norm_*).

GDN_FLAG_READ_ONLY = 4


_INT_MAX = 2 ** 31 - 1


def _ints(*sizes):
    """The C entry points count in 32-bit integers; ctypes would cut larger sizes off."""
    if max(sizes) > _INT_MAX:
        raise GdnError(f"a size above {_INT_MAX} is not supported")


def _cuda(t, name: str) -> int:
    """Index of the CUDA device that tensor ``t`` is on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GdnError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _dense(t, name: str, dtype, dev: int) -> int:
    """Pointer of a dense tensor on device ``dev``."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise GdnError(f"{name} must be a tensor on CUDA device {dev}")
    if t.dtype is not dtype:
        raise GdnError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise GdnError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name: str, dtype, dev: int):
    """Pointer and token stride of [tokens, ...] whose tokens are dense."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise GdnError(f"{name} must be a tensor on CUDA device {dev}")
    if t.dtype is not dtype:
        raise GdnError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if shape[0] > 1 and t.is_contiguous():
        return t.data_ptr(), t.stride(0)
    strides = t.stride()
    if len(shape) == 3 and shape[0] > 1 and strides[2] == 1 and strides[1] == shape[2]:
        return t.data_ptr(), strides[0]
    width = 1
    for i in range(len(shape) - 1, 0, -1):
        n = shape[i]
        if n != 1:
            if strides[i] != width:
                raise GdnError(f"{name}: the channels of a token must be contiguous")
            width *= n
    return t.data_ptr(), strides[0] if shape[0] > 1 else max(width, 1)


def _param(t, name: str, shape, dtype, dev: int):
    if t.shape != shape:
        raise GdnError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return _dense(t, name, dtype if t.dtype is dtype else torch.float32, dev)


def _call(dev: int, f, *args):
    """f(*args, stream of device ``dev``) with that device current."""
    if dev == torch._C._cuda_getDevice():
        return f(*args, torch._C._cuda_getCurrentRawStream(dev))
    with torch.cuda.device(dev):
        return f(*args, torch._C._cuda_getCurrentRawStream(dev))


def _like_parts(x, shapes):
    """New arrays of x's type and device, each of its own: views of one allocation would keep
    one another alive and share autograd's count of changes in place."""
    return tuple([x.new_empty(s) for s in shapes])


def _scratch(need: int, workspace, like, dev: int):
    """The workspace (a new one where none or too small a one is given), its pointer and its
    bytes.  The caller holds the tensor until the entry point has returned: an allocator may
    give the memory of one that nobody holds to another thread before the kernels are launched."""
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = like.new_empty(max(need, 16), dtype=torch.uint8)
    return (workspace, _dense(workspace, "workspace", workspace.dtype, dev),
            workspace.numel() * workspace.element_size())


def _sequences(cu_seqlens, slots, total, dev: int):
    """Pointers of the offsets and slots (int32 device tensors) and the number of sequences."""
    cu = sl = None
    N = total
    if cu_seqlens is not None:
        cu = _dense(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise GdnError("cu_seqlens must hold N + 1 offsets")
        N = cu_seqlens.shape[0] - 1
        _ints(N)
    if slots is not None:
        sl = _dense(slots, "slots", torch.int32, dev)
        if slots.shape != (N,):
            raise GdnError("slots must hold one slot per sequence")
    return cu, sl, N


def decode_runs(q, k, v, log_alpha, beta, states, slots=None, cu_seqlens=None, out=None,
                update: bool = True, l2norm_qk: bool = False, gate_logits: bool = False,
                want_output: bool = True):
    """Runs of tokens over a pool of states; returns o [total, Hv, Dv] (None without output).

    q, k [total, Hk, Dk], v [total, Hv, Dv] float32 or bfloat16 and log_alpha, beta
    [total, Hv] float32 may be slices of wider rows; Hv is a multiple of Hk (value
    head h reads key head h // (Hv // Hk)).  ``states`` [n_slots, Hv, Dv, Dk] float32
    is advanced in place, sequence n (tokens cu_seqlens[n] .. cu_seqlens[n + 1] - 1;
    None: one token each) in slot slots[n] (None: n).  ``cu_seqlens`` and ``slots`` are
    int32 tensors on q's device.  ``update=False`` leaves the states alone (outputs of
    a draft); ``want_output=False`` only advances them (q may be None).  A slot below 0
    marks a row of padding: output zero, no state.  Rows of no sequence are not written:
    they keep what ``out`` held.  ``l2norm_qk`` / ``gate_logits``: the
    input prologue, as in ``chunk_fwd``.
    """
    if not want_output and out is not None:
        raise GdnError("out without want_output")
    if want_output and q is None:
        raise GdnError("q is needed for the output")
    if k.dim() != 3 or v.dim() != 3 or v.shape[0] != k.shape[0] or (q is not None and
                                                                  q.shape != k.shape):
        raise GdnError("q, k must be [total,Hk,Dk] and v [total,Hv,Dv]")
    total, Hk, Dk = k.shape
    _, Hv, Dv = v.shape
    dev, dtype = _cuda(k, "k"), k.dtype
    code = _dtype_code(k)
    gates = (total, Hv)
    if log_alpha.shape != gates or beta.shape != gates:
        raise GdnError("log_alpha and beta must be [total,Hv]")
    if states.dim() != 4 or states.shape[1:] != (Hv, Dv, Dk):
        raise GdnError("states must be [n_slots,Hv,Dv,Dk]")
    if Hk == 0 or Hv % Hk:
        raise GdnError("Hv must be a multiple of Hk")
    n_slots = states.shape[0]
    _ints(total, Hk, Hv, Dk, Dv, n_slots)
    kp, ks = _rows(k, "k", dtype, dev)
    qp, qs = _rows(q, "q", dtype, dev) if q is not None else (None, 0)
    vp, vs = _rows(v, "v", dtype, dev)
    ap, as_ = _rows(log_alpha, "log_alpha", torch.float32, dev)
    bp, bs = _rows(beta, "beta", torch.float32, dev)
    cu, sl, N = _sequences(cu_seqlens, slots, total, dev)
    if slots is None and N > n_slots:
        raise GdnError("without slots, states must hold one state per sequence")
    o = op = None
    if want_output:
        o = out if out is not None else k.new_empty((total, Hv, Dv))
        if o.shape != (total, Hv, Dv):
            raise GdnError("out must be [total,Hv,Dv]")
        op = _dense(o, "out", dtype, dev)
    flags = _flags(l2norm_qk, gate_logits) | (0 if update else GDN_FLAG_READ_ONLY)
    _check(_call(dev, LIB.gdn_decode_runs, qp, kp, vp, ap, bp,
                 _dense(states, "states", torch.float32, dev), sl, cu, op, N, total, Hk, Hv, Dk,
                 Dv, n_slots, qs, ks, vs, as_, bs, code, flags), "gdn_decode_runs")
    return o


def _parts(tensors, splits, total, dtype, dev, name):
    """Pointers, strides and channel offsets (ctypes arrays) of the parts of y or dy."""
    ptrs, strides, begin = [], [], [0]
    for t, c in zip(tensors, splits):
        if t.shape != (total, c):
            raise GdnError(f"{name} must be [total,C], split as the channels are")
        p, s = _rows(t, name, dtype, dev)
        ptrs.append(p)
        strides.append(s)
        begin.append(begin[-1] + c)
    n = len(ptrs)
    return _PTRS[n](*ptrs), _LONGS[n](*strides), _INTS[n + 1](*begin)


_PTRS = [ctypes.c_void_p * n for n in range(4)]
_LONGS = [ctypes.c_longlong * n for n in range(4)]
_INTS = [ctypes.c_int * n for n in range(5)]


def short_conv_fwd(x, weight, bias=None, cu_seqlens=None, states=None, slots=None, silu: bool = True,
                   splits=None, out=None):
    """Short causal depthwise convolution over packed sequences: y [total, C].

    z[t] = bias + sum_j weight[:, j] * x[t - (W - 1) + j], y = silu(z) (or z).  x
    [total, C] float32 or bfloat16, possibly a slice of wider rows; weight [C, W], W in
    2..4, and bias [C] float32 or x's type.  ``splits``: up to three widths that sum to
    C; y is then a tuple of arrays of these widths (q, k and v from one call).
    ``states`` [n_slots, W - 1, C] in x's type: the last inputs of each sequence, used
    in front of it and always replaced; ``slots`` and ``cu_seqlens`` as in ``decode_runs``,
    except that the offsets must not decrease (valid sequences may then be left out).
    Without states sequences start from zero.  Rows of no sequence are not written: they
    keep what ``out`` held.
    """
    if x.dim() != 2 or weight.dim() != 2:
        raise GdnError("x must be [total,C] and weight [C,W]")
    total, C = x.shape
    W = weight.shape[1]
    dev, dtype = _cuda(x, "x"), x.dtype
    code = _dtype_code(x)
    xp, xs = _rows(x, "x", dtype, dev)
    wp = _param(weight, "weight", (C, W), dtype, dev)
    bp = None
    if bias is not None:
        if bias.dtype is not weight.dtype:
            raise GdnError("bias and weight must have one type")
        bp = _param(bias, "bias", (C,), dtype, dev)
    if slots is not None and states is None:
        raise GdnError("slots without states")
    cu, sl, N = _sequences(cu_seqlens, slots, total, dev)
    sp, n_slots = None, 0
    if states is not None:
        if states.dim() != 3 or states.shape[1:] != (W - 1, C):
            raise GdnError("states must be [n_slots,W-1,C]")
        n_slots = states.shape[0]
        if slots is None and N > n_slots:
            raise GdnError("without slots, states must hold one state per sequence")
        sp = _dense(states, "states", dtype, dev)
    _ints(total, C, W, n_slots)
    widths = [C] if splits is None else list(splits)
    if not 1 <= len(widths) <= 3 or sum(widths) != C or min(widths) <= 0:
        raise GdnError("splits must be one to three widths that sum to C")
    n = len(widths)
    if out is None:
        ys = _like_parts(x, [(total, c) for c in widths])
        ptrs, strides = _PTRS[n](*[y.data_ptr() for y in ys]), _LONGS[n](*widths)
        begin = _INTS[n + 1](0, *accumulate(widths))
    else:
        ys = (out,) if splits is None else tuple(out)
        if len(ys) != n:
            raise GdnError("out must hold one array per split")
        ptrs, strides, begin = _parts(ys, widths, total, dtype, dev, "out")
    st = _call(dev, LIB.gdn_short_conv_fwd, xp, wp, bp, sp, sl, cu, ptrs, strides, begin,
               len(widths), N, total, C, W, n_slots, xs, int(silu), code, _dtype_code(weight))
    _check(st, "gdn_short_conv_fwd")
    return ys[0] if splits is None else ys


def short_conv_bwd_workspace_size(total: int, C: int, W: int) -> int:
    return int(LIB.gdn_short_conv_bwd_workspace_size(total, C, W))


def short_conv_bwd(dy, x, weight, bias=None, cu_seqlens=None, silu: bool = True, workspace=None):
    """Gradients of ``short_conv_fwd`` for sequences that start from zero.

    ``dy`` [total, C] or a tuple of the parts' gradients; the rest as in the forward.
    Returns (dx [total, C] in x's type, dweight [C, W] float32, dbias [C] float32 or
    None without bias).
    """
    if x.dim() != 2 or weight.dim() != 2:
        raise GdnError("x must be [total,C] and weight [C,W]")
    total, C = x.shape
    W = weight.shape[1]
    dev, dtype = _cuda(x, "x"), x.dtype
    code = _dtype_code(x)
    xp, xs = _rows(x, "x", dtype, dev)
    wp = _param(weight, "weight", (C, W), dtype, dev)
    bp = None
    if bias is not None:
        if bias.dtype is not weight.dtype:
            raise GdnError("bias and weight must have one type")
        bp = _param(bias, "bias", (C,), dtype, dev)
    _ints(total, C, W)
    cu, _, N = _sequences(cu_seqlens, None, total, dev)
    dys = (dy,) if isinstance(dy, torch.Tensor) else tuple(dy)
    widths = [d.shape[1] for d in dys if d.dim() == 2]
    if not 1 <= len(dys) <= 3 or len(widths) != len(dys) or sum(widths) != C:
        raise GdnError("dy must be [total,C] or up to three arrays of C channels in all")
    ptrs, strides, begin = _parts(dys, widths, total, dtype, dev, "dy")
    dx = x.new_empty((total, C))
    dw = x.new_empty((C, W), dtype=torch.float32)
    db = x.new_empty((C,), dtype=torch.float32) if bias is not None else None
    workspace, ws, nbytes = _scratch(LIB.gdn_short_conv_bwd_workspace_size(total, C, W), workspace,
                                     x, dev)
    st = _call(dev, LIB.gdn_short_conv_bwd, ptrs, strides, begin, len(dys), xp, wp, bp, cu,
               dx.data_ptr(), dw.data_ptr(), db.data_ptr() if db is not None else None, N, total,
               C, W, xs, int(silu), code, _dtype_code(weight), ws, nbytes)
    _check(st, "gdn_short_conv_bwd")
    return dx, dw, db


def _norm_rows(t, name, shape, dtype, dev):
    """Pointer and token stride of a [..., D] tensor: its last axis but one counts the heads
    of a token where there are three axes or more, the axes before it the tokens."""
    if t.shape != shape:
        raise GdnError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if len(shape) == 1:
        t = t.unsqueeze(0)
    elif len(shape) > 3:
        try:
            t = t.view(-1, *t.shape[-2:])
        except RuntimeError:
            raise GdnError(f"{name}: its leading axes must be contiguous with one another") from None
    return _rows(t, name, dtype, dev)


def _norm_sizes(shape):
    if len(shape) < 1 or shape[-1] < 1:
        raise GdnError("x must be [...,D] with D >= 1")
    heads = shape[-2] if len(shape) > 2 else 1
    tokens = 1
    for n in shape[:-2] if len(shape) > 2 else shape[:-1]:
        tokens *= n
    _ints(tokens, heads, shape[-1])
    return tokens, heads, shape[-1]


def rms_norm_fwd(x, weight, residual=None, gate=None, eps: float = 1e-6, quant=None, out=None,
                 h_out=None):
    """Root-mean-square norm over the last axis: returns (y, scale, h).

    h = x + residual, rounded to x's type (h is None and x is used without residual);
    y = h / sqrt(mean h^2 + eps) * weight (* silu(gate)).  x, residual and gate [..., D]
    float32 or bfloat16, with three axes or more the last but one being a token's
    heads; tokens may be slices of wider rows.  weight [D] float32 or x's type.
    ``quant``: None: y in x's type; "row" or "group": y in float8_e4m3fn, with ``scale``
    [..., D / group] float32 per row or per 128 columns, the value being y * scale.
    ``out`` / ``h_out``: arrays for y and h (h_out may be the residual itself).
    """
    shape, dev, dtype = x.shape, _cuda(x, "x"), x.dtype
    code = _dtype_code(x)
    tokens, heads, D = _norm_sizes(shape)
    xp, xs = _norm_rows(x, "x", shape, dtype, dev)
    wp = _param(weight, "weight", (D,), dtype, dev)
    rp, rs = _norm_rows(residual, "residual", shape, dtype, dev) if residual is not None else (None, 0)
    gp, gs = _norm_rows(gate, "gate", shape, dtype, dev) if gate is not None else (None, 0)
    if quant not in (None, "row", "group"):
        raise GdnError('quant must be None, "row" or "group"')
    group = 0 if quant is None else D if quant == "row" else 128
    if quant == "group" and D % 128:
        raise GdnError("groups of 128 columns need D to be a multiple of 128")
    ytype = dtype if quant is None else torch.float8_e4m3fn
    y = out if out is not None else x.new_empty(shape, dtype=ytype)
    if y.shape != shape:
        raise GdnError("out must be shaped like x")
    yp = _dense(y, "out", ytype, dev)
    scale = sc = None
    if group:
        scale = x.new_empty(shape[:-1] + (D // group,), dtype=torch.float32)
        sc = scale.data_ptr()
    h = hp = None
    if residual is not None:
        h = h_out if h_out is not None else x.new_empty(shape)
        if h.shape != shape:
            raise GdnError("h_out must be shaped like x")
        hp = _dense(h, "h_out", dtype, dev)
    elif h_out is not None:
        raise GdnError("h_out without residual")
    st = _call(dev, LIB.gdn_rms_norm_fwd, xp, wp, rp, gp, yp, sc, hp, tokens, heads, D, group, xs,
               rs, gs, eps, code, _dtype_code(weight))
    _check(st, "gdn_rms_norm_fwd")
    return y, scale, h


def rms_norm_bwd_workspace_size(tokens: int, heads: int, D: int) -> int:
    return int(LIB.gdn_rms_norm_bwd_workspace_size(tokens, heads, D))


def rms_norm_bwd(dy, x, weight, gate=None, d_res=None, eps: float = 1e-6, workspace=None):
    """Gradients of ``rms_norm_fwd``: returns (dx, dweight, dgate).

    ``x`` is the forward's x, or its h where there was a residual; ``dy`` the gradient of
    y (of the values it stands for, where it is held in 8 bits); ``d_res`` that of h, if
    h is used again.  dx, in x's type, is the gradient of both x and the residual;
    dweight [D] is float32; dgate is None without gate.
    """
    shape, dev, dtype = x.shape, _cuda(x, "x"), x.dtype
    code = _dtype_code(x)
    tokens, heads, D = _norm_sizes(shape)
    xp, xs = _norm_rows(x, "x", shape, dtype, dev)
    yp, ys = _norm_rows(dy, "dy", shape, dtype, dev)
    wp = _param(weight, "weight", (D,), dtype, dev)
    gp, gs = _norm_rows(gate, "gate", shape, dtype, dev) if gate is not None else (None, 0)
    dp, ds = _norm_rows(d_res, "d_res", shape, dtype, dev) if d_res is not None else (None, 0)
    dx, dgate = _like_parts(x, (shape, shape)) if gate is not None else (x.new_empty(shape), None)
    dw = x.new_empty((D,), dtype=torch.float32)
    workspace, ws, nbytes = _scratch(LIB.gdn_rms_norm_bwd_workspace_size(tokens, heads, D), workspace,
                                     x, dev)
    st = _call(dev, LIB.gdn_rms_norm_bwd, yp, xp, wp, gp, dp, dx.data_ptr(), dw.data_ptr(),
               dgate.data_ptr() if dgate is not None else None, tokens, heads, D, ys, xs, gs, ds,
               eps, code, _dtype_code(weight), ws, nbytes)
    _check(st, "gdn_rms_norm_bwd")
    return dx, dw, dgate
