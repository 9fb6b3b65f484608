"""ctypes binding of liborthros.so (the C ABI declared in include/orthros.h).

Only argument marshalling happens here: shapes and strides are read off torch
tensors, device pointers and the current CUDA stream are handed to the C entry
points, and a non-OK status becomes an exception.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "_lib", "liborthros.so")

DEVERR_POSITION = 1
DEVERR_CACHE_FULL = 2
DEVERR_TIMEOUT = 4
DEVERR_RANGE = 8

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration",
           3: "workspace missing or too small", 4: "CUDA error"}


class OrthrosError(RuntimeError):
    pass


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load liborthros.so (built by build.py / __graft_entry__.build()); raise if missing."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(library_path):
                raise OrthrosError(
                    f"{library_path} is missing: build it with "
                    "`python -m long_context_attention_orthros_gb300.build`")
            L = ctypes.CDLL(library_path)
            P, I, F, L64, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64,
                                ctypes.c_size_t)
            L.orthros_status_string.restype = ctypes.c_char_p
            L.orthros_status_string.argtypes = [I]
            L.orthros_version.restype = I
            L.orthros_swa_fwd.restype = I
            L.orthros_swa_fwd.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, L64, L64, L64, P, P]
            L.orthros_swa_fwd_rows.restype = I
            L.orthros_swa_fwd_rows.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, L64, L64, L64, I, I, P, P]
            L.orthros_xattn_workspace_size.restype = SZ
            L.orthros_xattn_workspace_size.argtypes = [I, I, I, I, I, I]
            L.orthros_xattn_fwd.restype = I
            L.orthros_xattn_fwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, L64, L64, L64,
                                            P, SZ, P, P]
            L.orthros_prefill_workspace_size.restype = SZ
            L.orthros_prefill_workspace_size.argtypes = [I, I, I, I, I, I]
            L.orthros_prefill_fwd.restype = I
            L.orthros_prefill_fwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F,
                                              L64, L64, L64, L64, L64, P, SZ, P, P]
            L.orthros_decode_workspace_size.restype = SZ
            L.orthros_decode_workspace_size.argtypes = [I, I, I, I, I]
            L.orthros_decode_step.restype = I
            L.orthros_decode_step.argtypes = [P, P, P, P, P, P, P, I, P, P, P, P, P, P, I, I, I, I,
                                              I, F, P, SZ, P, P]
            L.orthros_swa_bwd_workspace_size.restype = SZ
            L.orthros_swa_bwd_workspace_size.argtypes = [I, I, I, I, I]
            L.orthros_swa_bwd.restype = I
            L.orthros_swa_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P,
                                          SZ, P, P]
            L.orthros_swa_fwd_lse.restype = I
            L.orthros_swa_fwd_lse.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, L64, L64, L64, P, P]
            L.orthros_xattn_bwd_workspace_size.restype = SZ
            L.orthros_xattn_bwd_workspace_size.argtypes = [I, I, I, I, I, I]
            L.orthros_xattn_bwd.restype = I
            L.orthros_xattn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F,
                                            I, P, SZ, P, P]
            L.orthros_attn_bwd_workspace_size.restype = SZ
            L.orthros_attn_bwd_workspace_size.argtypes = [I, I, I, I, I, I]
            L.orthros_attn_bwd.restype = I
            L.orthros_attn_bwd.argtypes = [P] * 23 + [I, I, I, I, I, I, I, F, P, SZ, P, P]
            L.orthros_xattn_fwd_lse.restype = I
            L.orthros_xattn_fwd_lse.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, L64, L64, L64,
                                                P, SZ, P, P]
            L.orthros_kv_quantize.restype = I
            L.orthros_kv_quantize.argtypes = [P] * 8 + [I] * 6 + [L64, P, P]
            L.orthros_kv_dequantize.restype = I
            L.orthros_kv_dequantize.argtypes = [P] * 8 + [I] * 6 + [L64, P, P]
            L.orthros_decode_q8_workspace_size.restype = SZ
            L.orthros_decode_q8_workspace_size.argtypes = [I] * 5
            L.orthros_decode_step_q8.restype = I
            L.orthros_decode_step_q8.argtypes = [P] * 9 + [I, I] + [P] * 6 + [I] * 5 + [F, P, SZ, P, P]
            L.orthros_decode_prefix_workspace_size.restype = SZ
            L.orthros_decode_prefix_workspace_size.argtypes = [I] * 6
            L.orthros_decode_step_prefix.restype = I
            L.orthros_decode_step_prefix.argtypes = [P] * 6 + [I, P, P, P, I] + [P] * 6 + [I] * 5 + [F, P, SZ, P, P]
            L.orthros_xattn_prefix_workspace_size.restype = SZ
            L.orthros_xattn_prefix_workspace_size.argtypes = [I] * 7
            L.orthros_xattn_prefix_fwd.restype = I
            L.orthros_xattn_prefix_fwd.argtypes = [P] * 4 + [I] + [P] * 5 + [I] * 6 + [F, L64, L64, L64, P, SZ, P, P]
            L.orthros_swa_sink_fwd.restype = I
            L.orthros_swa_sink_fwd.argtypes = [P] * 7 + [I] * 7 + [F, L64, L64, L64, I, I, P, P]
            L.orthros_swa_sink_bwd_workspace_size.restype = SZ
            L.orthros_swa_sink_bwd_workspace_size.argtypes = [I] * 5
            L.orthros_swa_sink_bwd.restype = I
            L.orthros_swa_sink_bwd.argtypes = [P] * 13 + [I] * 7 + [F, P, SZ, P, P]
            L.orthros_decode_tree_workspace_size.restype = SZ
            L.orthros_decode_tree_workspace_size.argtypes = [I] * 6
            L.orthros_decode_tree.restype = I
            L.orthros_decode_tree.argtypes = [P] * 9 + [I] + [P] * 6 + [I] * 7 + [F, P, SZ, P, P]
            L.orthros_decode_tree_accept.restype = I
            L.orthros_decode_tree_accept.argtypes = [P] * 7 + [I, P] + [I] * 4 + [P, P]
            L.orthros_decode_tree_accept_nodes.restype = I
            L.orthros_decode_tree_accept_nodes.argtypes = [P] * 8 + [I, P] + [I] * 4 + [P, P]
            _lib = L
    return _lib


def _check(status: int, what: str) -> None:
    if status != 0:
        raise OrthrosError(f"{what}: {_STATUS.get(status, status)}")


def _ptr(t):
    """Device pointer of a tensor argument.  Every pointer the library takes is a device
    pointer of the call's GPU (the current device inside the calls below): a host tensor or
    one on another GPU is refused here rather than handed to a kernel."""
    if t is None:
        return None
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise OrthrosError(f"tensor arguments must be CUDA tensors on the call's device (got {t.device})")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _bf16_rows(t: torch.Tensor, name: str) -> int:
    """Check a [B, T, H, d] bf16 CUDA tensor whose (T, H, d) block is dense; return its batch stride."""
    if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 4:
        raise OrthrosError(f"{name} must be a 4-D bf16 CUDA tensor [B, T, H, d]")
    B, T, H, d = t.shape
    # strides of size-1 dimensions are irrelevant (numpy/torch may report anything there)
    if ((d > 1 and t.stride(3) != 1) or (H > 1 and t.stride(2) != d)
            or (T > 1 and t.stride(1) != H * d)):
        raise OrthrosError(f"{name}: the [T, H, d] part must be dense (d contiguous)")
    # an expanded batch: the library takes a batch stride of 0 for the dense one
    if B > 1 and t.stride(0) == 0 and T * H * d > 0:
        raise OrthrosError(f"{name}: the sequences of a batch must not be one another's memory (expanded tensor)")
    return t.stride(0) if B > 1 else T * H * d


def _vec(t: torch.Tensor, name: str, Hq: int, d: int) -> None:
    if t.dtype != torch.float32 or not t.is_cuda or tuple(t.shape) != (Hq, d) or not t.is_contiguous():
        raise OrthrosError(f"{name} must be a contiguous fp32 CUDA tensor [Hq, d]")


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def swa_fwd(q_raw, k, v, alpha, beta, window: int = 128, scale=None, out=None, dev_err=None):
    """Eq. (4): o[b, t] = softmax over keys max(0, t-window+1)..t of (q . k) * scale, applied to v,
    with q = q_raw * alpha + beta.  q_raw [B, Tq, Hq, d] (Tq >= T, only the first T rows are
    read, so copies may be appended after the base tokens); k, v [B, T, Hkv, d]."""
    B, T, Hkv, d = k.shape
    Hq = q_raw.shape[2]
    qs = _bf16_rows(q_raw, "q_raw")
    ks = _bf16_rows(k, "k")
    if _bf16_rows(v, "v") != ks or v.shape != k.shape:
        raise OrthrosError("k and v must have the same shape and strides")
    if q_raw.shape[0] != B or q_raw.shape[1] < T or q_raw.shape[3] != d:
        raise OrthrosError("q_raw shape does not match k")
    _vec(alpha, "alpha", Hq, d)
    _vec(beta, "beta", Hq, d)
    if out is None:
        out = torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=k.device)
    os_ = _bf16_rows(out, "out")
    with torch.cuda.device(k.device):
        st = lib().orthros_swa_fwd(_ptr(q_raw), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(out),
                                   B, T, Hq, Hkv, d, int(window), _scale(scale, d), qs, ks, os_,
                                   _ptr(dev_err), _stream(k.device))
    _check(st, "orthros_swa_fwd")
    return out


def swa_fwd_rows(q_raw, k, v, alpha, beta, row_begin: int, row_end: int, window: int = 128, scale=None,
                 out=None, dev_err=None):
    """swa_fwd for output rows row_begin..row_end-1 of every sequence only (chunked prefill);
    other rows of `out` are left as they are.  row_begin a multiple of 128, row_end a multiple
    of 128 or T.  Keys are read from row max(0, row_begin - window + 1)."""
    B, T, Hkv, d = k.shape
    Hq = q_raw.shape[2]
    qs = _bf16_rows(q_raw, "q_raw")
    ks = _bf16_rows(k, "k")
    if _bf16_rows(v, "v") != ks or v.shape != k.shape:
        raise OrthrosError("k and v must have the same shape and strides")
    if q_raw.shape[0] != B or q_raw.shape[1] < T or q_raw.shape[3] != d:
        raise OrthrosError("q_raw shape does not match k")
    _vec(alpha, "alpha", Hq, d)
    _vec(beta, "beta", Hq, d)
    if out is None:
        out = torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=k.device)
    os_ = _bf16_rows(out, "out")
    with torch.cuda.device(k.device):
        st = lib().orthros_swa_fwd_rows(_ptr(q_raw), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(out),
                                        B, T, Hq, Hkv, d, int(window), _scale(scale, d), qs, ks, os_,
                                        int(row_begin), int(row_end), _ptr(dev_err), _stream(k.device))
    _check(st, "orthros_swa_fwd_rows")
    return out


def xattn_workspace_size(B, T_out, T_kv, Hq, Hkv, d) -> int:
    return int(lib().orthros_xattn_workspace_size(B, T_out, T_kv, Hq, Hkv, d))


def decode_workspace_size(B, L_max, Hq, Hkv, d) -> int:
    return int(lib().orthros_decode_workspace_size(B, L_max, Hq, Hkv, d))


def xattn_fwd(qc_raw, pos, k, v, alpha_c, beta_c, scale=None, out=None, workspace=None, dev_err=None,
              lse=None):
    """Eq. (5): copy i of sequence b at original position pos[b, i] attends over k/v rows
    0..pos[b, i].  qc_raw [B, T_out, Hq, d] (may be a view of an appended buffer);
    pos int32 [B, T_out]; k, v [B, T_kv, Hkv, d].  With lse (fp32 [B, T_out, Hq], or True for
    a fresh one) each copy row's log-sum-exp is written too, for xattn_bwd, and (out, lse)
    is returned."""
    B, T_kv, Hkv, d = k.shape
    T_out, Hq = qc_raw.shape[1], qc_raw.shape[2]
    qs = _bf16_rows(qc_raw, "qc_raw")
    ks = _bf16_rows(k, "k")
    if _bf16_rows(v, "v") != ks or v.shape != k.shape:
        raise OrthrosError("k and v must have the same shape and strides")
    if pos.dtype != torch.int32 or tuple(pos.shape) != (B, T_out) or not pos.is_contiguous():
        raise OrthrosError("pos must be a contiguous int32 tensor [B, T_out]")
    _vec(alpha_c, "alpha_c", Hq, d)
    _vec(beta_c, "beta_c", Hq, d)
    if out is None:
        out = torch.empty((B, T_out, Hq, d), dtype=torch.bfloat16, device=k.device)
    os_ = _bf16_rows(out, "out")
    need = xattn_workspace_size(B, T_out, T_kv, Hq, Hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=k.device)
    if lse is True:
        lse = torch.empty((B, T_out, Hq), dtype=torch.float32, device=k.device)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, T_out, Hq) or
                            not lse.is_contiguous()):
        raise OrthrosError("lse must be a contiguous fp32 tensor [B, T_out, Hq]")
    with torch.cuda.device(k.device):
        if lse is None:
            st = lib().orthros_xattn_fwd(_ptr(qc_raw), _ptr(pos), _ptr(k), _ptr(v), _ptr(alpha_c),
                                         _ptr(beta_c), _ptr(out), B, T_out, T_kv, Hq, Hkv, d,
                                         _scale(scale, d), qs, ks, os_, _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _ptr(dev_err),
                                         _stream(k.device))
        else:
            st = lib().orthros_xattn_fwd_lse(_ptr(qc_raw), _ptr(pos), _ptr(k), _ptr(v), _ptr(alpha_c),
                                             _ptr(beta_c), _ptr(out), _ptr(lse), B, T_out, T_kv, Hq, Hkv, d,
                                             _scale(scale, d), qs, ks, os_, _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _ptr(dev_err),
                                             _stream(k.device))
    _check(st, "orthros_xattn_fwd")
    return out if lse is None else (out, lse)


def prefill_workspace_size(B, T, T_out, Hq, Hkv, d) -> int:
    return int(lib().orthros_prefill_workspace_size(B, T, T_out, Hq, Hkv, d))


def prefill_fwd(q_raw, k, v, alpha, beta, qc_raw, pos, alpha_c, beta_c, window: int = 128, scale=None,
                out=None, out_c=None, workspace=None, dev_err=None):
    """One prefill layer in one call: swa_fwd for the base stream, then xattn_fwd (T_kv = T)
    for the output copies.  Returns (o, oc)."""
    B, T, Hkv, d = k.shape
    Hq = q_raw.shape[2]
    T_out = qc_raw.shape[1]
    qs = _bf16_rows(q_raw, "q_raw")
    qcs = _bf16_rows(qc_raw, "qc_raw")
    ks = _bf16_rows(k, "k")
    if _bf16_rows(v, "v") != ks or v.shape != k.shape:
        raise OrthrosError("k and v must have the same shape and strides")
    if q_raw.shape[0] != B or q_raw.shape[1] < T or q_raw.shape[3] != d:
        raise OrthrosError("q_raw shape does not match k")
    if qc_raw.shape[0] != B or qc_raw.shape[2] != Hq or qc_raw.shape[3] != d:
        raise OrthrosError("qc_raw shape does not match q_raw")
    if pos.dtype != torch.int32 or tuple(pos.shape) != (B, T_out) or not pos.is_contiguous():
        raise OrthrosError("pos must be a contiguous int32 tensor [B, T_out]")
    for t, nm in ((alpha, "alpha"), (beta, "beta"), (alpha_c, "alpha_c"), (beta_c, "beta_c")):
        _vec(t, nm, Hq, d)
    if out is None:
        out = torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=k.device)
    if out_c is None:
        out_c = torch.empty((B, T_out, Hq, d), dtype=torch.bfloat16, device=k.device)
    os_ = _bf16_rows(out, "out")
    ocs = _bf16_rows(out_c, "out_c")
    if workspace is None:
        workspace = torch.empty(max(prefill_workspace_size(B, T, T_out, Hq, Hkv, d), 256),
                                dtype=torch.uint8, device=k.device)
    with torch.cuda.device(k.device):
        st = lib().orthros_prefill_fwd(_ptr(q_raw), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(out),
                                       _ptr(qc_raw), _ptr(pos), _ptr(alpha_c), _ptr(beta_c), _ptr(out_c),
                                       B, T, T_out, Hq, Hkv, d, int(window), _scale(scale, d), qs, ks, os_,
                                       qcs, ocs, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _ptr(dev_err), _stream(k.device))
    _check(st, "orthros_prefill_fwd")
    return out, out_c


def swa_bwd_workspace_size(B, T, Hq, Hkv, d) -> int:
    return int(lib().orthros_swa_bwd_workspace_size(B, T, Hq, Hkv, d))


def swa_fwd_lse(q_raw, k, v, alpha, beta, window: int = 128, scale=None, out=None, lse=None, dev_err=None):
    """swa_fwd that also returns each row's log-sum-exp, fp32 [B, T, Hq] (natural log of the
    softmax normaliser), for swa_bwd.  Returns (o, lse)."""
    B, T, Hkv, d = k.shape
    Hq = q_raw.shape[2]
    qs = _bf16_rows(q_raw, "q_raw")
    ks = _bf16_rows(k, "k")
    if _bf16_rows(v, "v") != ks or v.shape != k.shape:
        raise OrthrosError("k and v must have the same shape and strides")
    if q_raw.shape[0] != B or q_raw.shape[1] < T or q_raw.shape[3] != d:
        raise OrthrosError("q_raw shape does not match k")
    _vec(alpha, "alpha", Hq, d)
    _vec(beta, "beta", Hq, d)
    if out is None:
        out = torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=k.device)
    if lse is None:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=k.device)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, T, Hq) or not lse.is_contiguous():
        raise OrthrosError("lse must be a contiguous fp32 tensor [B, T, Hq]")
    os_ = _bf16_rows(out, "out")
    with torch.cuda.device(k.device):
        st = lib().orthros_swa_fwd_lse(_ptr(q_raw), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(out), _ptr(lse),
                                       B, T, Hq, Hkv, d, int(window), _scale(scale, d), qs, ks, os_, _ptr(dev_err),
                                       _stream(k.device))
    _check(st, "orthros_swa_fwd_lse")
    return out, lse


def swa_bwd(q_raw, k, v, alpha, beta, o, dO, window: int = 128, scale=None, workspace=None, dev_err=None,
            lse=None):
    """Gradient of Eq. (4) with its scale-offset: returns fp32 (dq_raw, dk, dv, dalpha, dbeta) for
    the output gradient dO, given the forward inputs and the forward output o.  q_raw, o, dO
    [B, T, Hq, d] and k, v [B, T, Hkv, d], all dense bf16; alpha, beta [Hq, d] fp32."""
    B, T, Hkv, d = k.shape
    Hq = q_raw.shape[2]
    for t, nm, shp in ((q_raw, "q_raw", (B, T, Hq, d)), (o, "o", (B, T, Hq, d)), (dO, "dO", (B, T, Hq, d)),
                       (k, "k", (B, T, Hkv, d)), (v, "v", (B, T, Hkv, d))):
        if t.dtype != torch.bfloat16 or not t.is_cuda or tuple(t.shape) != shp or not t.is_contiguous():
            raise OrthrosError(f"{nm} must be a contiguous bf16 CUDA tensor {shp}")
    _vec(alpha, "alpha", Hq, d)
    _vec(beta, "beta", Hq, d)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, T, Hq) or not lse.is_contiguous()):
        raise OrthrosError("lse must be a contiguous fp32 tensor [B, T, Hq] (from swa_fwd_lse)")
    f32 = dict(dtype=torch.float32, device=k.device)
    dq = torch.empty((B, T, Hq, d), **f32)
    dk = torch.empty((B, T, Hkv, d), **f32)
    dv = torch.empty((B, T, Hkv, d), **f32)
    dalpha = torch.empty((Hq, d), **f32)
    dbeta = torch.empty((Hq, d), **f32)
    if workspace is None:
        workspace = torch.empty(max(swa_bwd_workspace_size(B, T, Hq, Hkv, d), 256), dtype=torch.uint8,
                                device=k.device)
    with torch.cuda.device(k.device):
        st = lib().orthros_swa_bwd(_ptr(q_raw), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o), _ptr(dO),
                                   _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dalpha), _ptr(dbeta), B, T, Hq, Hkv, d,
                                   int(window), _scale(scale, d), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(dev_err), _stream(k.device))
    _check(st, "orthros_swa_bwd")
    return dq, dk, dv, dalpha, dbeta


def xattn_bwd_workspace_size(B, T_out, T_kv, Hq, Hkv, d) -> int:
    return int(lib().orthros_xattn_bwd_workspace_size(B, T_out, T_kv, Hq, Hkv, d))


def xattn_bwd(qc_raw, pos, k, v, alpha_c, beta_c, oc, dOc, scale=None, dk=None, dv=None, workspace=None,
              dev_err=None, lse=None):
    """Gradient of Eq. (5) with the copies' scale-offset: returns fp32 (dqc_raw, dk, dv, dalpha_c,
    dbeta_c).  Passing dk, dv (fp32 [B, T_kv, Hkv, d], e.g. from swa_bwd) adds the copies' share
    to them in place; otherwise fresh tensors hold the copies' share alone.  qc_raw, oc, dOc
    [B, T_out, Hq, d] and k, v [B, T_kv, Hkv, d] dense bf16; pos int32 [B, T_out]; lse (optional)
    the forward's fp32 [B, T_out, Hq] log-sum-exp (xattn_fwd with lse)."""
    B, T_kv, Hkv, d = k.shape
    T_out, Hq = qc_raw.shape[1], qc_raw.shape[2]
    for t, nm, shp in ((qc_raw, "qc_raw", (B, T_out, Hq, d)), (oc, "oc", (B, T_out, Hq, d)),
                       (dOc, "dOc", (B, T_out, Hq, d)), (k, "k", (B, T_kv, Hkv, d)), (v, "v", (B, T_kv, Hkv, d))):
        if t.dtype != torch.bfloat16 or not t.is_cuda or tuple(t.shape) != shp or not t.is_contiguous():
            raise OrthrosError(f"{nm} must be a contiguous bf16 CUDA tensor {shp}")
    if pos.dtype != torch.int32 or tuple(pos.shape) != (B, T_out) or not pos.is_contiguous():
        raise OrthrosError("pos must be a contiguous int32 tensor [B, T_out]")
    _vec(alpha_c, "alpha_c", Hq, d)
    _vec(beta_c, "beta_c", Hq, d)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, T_out, Hq) or
                            not lse.is_contiguous()):
        raise OrthrosError("lse must be a contiguous fp32 tensor [B, T_out, Hq]")
    f32 = dict(dtype=torch.float32, device=k.device)
    accumulate = dk is not None
    if (dk is None) != (dv is None):
        raise OrthrosError("pass both dk and dv, or neither")
    for t, nm in ((dk, "dk"), (dv, "dv")):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (B, T_kv, Hkv, d)
                              or not t.is_contiguous()):
            raise OrthrosError(f"{nm} must be a contiguous fp32 tensor [B, T_kv, Hkv, d]")
    if not accumulate:
        dk = torch.empty((B, T_kv, Hkv, d), **f32)
        dv = torch.empty((B, T_kv, Hkv, d), **f32)
    dq = torch.empty((B, T_out, Hq, d), **f32)
    dalpha = torch.empty((Hq, d), **f32)
    dbeta = torch.empty((Hq, d), **f32)
    if workspace is None:
        workspace = torch.empty(max(xattn_bwd_workspace_size(B, T_out, T_kv, Hq, Hkv, d), 256), dtype=torch.uint8,
                                device=k.device)
    with torch.cuda.device(k.device):
        st = lib().orthros_xattn_bwd(_ptr(qc_raw), _ptr(pos), _ptr(k), _ptr(v), _ptr(alpha_c), _ptr(beta_c),
                                     _ptr(oc), _ptr(dOc), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dalpha),
                                     _ptr(dbeta),
                                     B, T_out, T_kv, Hq, Hkv, d, _scale(scale, d), int(accumulate),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _ptr(dev_err), _stream(k.device))
    _check(st, "orthros_xattn_bwd")
    return dq, dk, dv, dalpha, dbeta


def attn_bwd_workspace_size(B, T, T_out, Hq, Hkv, d) -> int:
    return int(lib().orthros_attn_bwd_workspace_size(B, T, T_out, Hq, Hkv, d))


def attn_bwd(q_raw, k, v, alpha, beta, o, dO, qc_raw, pos, alpha_c, beta_c, oc, dOc, window: int = 128,
             scale=None, lse=None, lsec=None, workspace=None, dev_err=None):
    """A layer's attention gradient, both streams in one call: returns fp32 (dq_raw, dk, dv, dalpha,
    dbeta, dqc_raw, dalpha_c, dbeta_c), dk and dv holding both streams' shares.  Base tensors as
    swa_bwd, copy tensors as xattn_bwd (T_kv = T); lse / lsec the forwards' log-sum-exp or None."""
    B, T, Hkv, d = k.shape
    Hq, T_out = q_raw.shape[2], qc_raw.shape[1]
    for t, nm, shp in ((q_raw, "q_raw", (B, T, Hq, d)), (o, "o", (B, T, Hq, d)), (dO, "dO", (B, T, Hq, d)),
                       (qc_raw, "qc_raw", (B, T_out, Hq, d)), (oc, "oc", (B, T_out, Hq, d)),
                       (dOc, "dOc", (B, T_out, Hq, d)), (k, "k", (B, T, Hkv, d)), (v, "v", (B, T, Hkv, d))):
        if t.dtype != torch.bfloat16 or not t.is_cuda or tuple(t.shape) != shp or not t.is_contiguous():
            raise OrthrosError(f"{nm} must be a contiguous bf16 CUDA tensor {shp}")
    if pos.dtype != torch.int32 or tuple(pos.shape) != (B, T_out) or not pos.is_contiguous():
        raise OrthrosError("pos must be a contiguous int32 tensor [B, T_out]")
    for t, nm in ((alpha, "alpha"), (beta, "beta"), (alpha_c, "alpha_c"), (beta_c, "beta_c")):
        _vec(t, nm, Hq, d)
    for t, nm, shp in ((lse, "lse", (B, T, Hq)), (lsec, "lsec", (B, T_out, Hq))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shp or not t.is_contiguous()):
            raise OrthrosError(f"{nm} must be a contiguous fp32 tensor {shp}")
    f32 = dict(dtype=torch.float32, device=k.device)
    out = [torch.empty(shp, **f32) for shp in ((B, T, Hq, d), (B, T, Hkv, d), (B, T, Hkv, d), (Hq, d), (Hq, d),
                                                (B, T_out, Hq, d), (Hq, d), (Hq, d))]
    if workspace is None:
        workspace = torch.empty(attn_bwd_workspace_size(B, T, T_out, Hq, Hkv, d), dtype=torch.uint8,
                                device=k.device)
    with torch.cuda.device(k.device):
        st = lib().orthros_attn_bwd(_ptr(q_raw), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o), _ptr(dO),
                                    _ptr(lse), _ptr(qc_raw), _ptr(pos), _ptr(alpha_c), _ptr(beta_c), _ptr(oc),
                                    _ptr(dOc), _ptr(lsec), *[_ptr(t) for t in out], B, T, T_out, Hq, Hkv, d,
                                    int(window), _scale(scale, d), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _ptr(dev_err),
                                    _stream(k.device))
    _check(st, "orthros_attn_bwd")
    return tuple(out)


def decode_workspace(B, L_max, Hq, Hkv, d, device) -> torch.Tensor:
    """A zero-filled workspace for decode_step (reusable step after step)."""
    return torch.zeros(max(decode_workspace_size(B, L_max, Hq, Hkv, d), 256), dtype=torch.uint8,
                       device=device)


def decode_step(q_new, qc_new, k_new, v_new, k_cache, v_cache, cache_len, alpha, beta, alpha_c,
                beta_c, window: int = 128, scale=None, o=None, oc=None, workspace=None, dev_err=None):
    """One decode step: append k_new/v_new at row cache_len[b], base SWA for q_new, full-cache
    attention for the copy qc_new, then cache_len += 1.  q_new, qc_new [B, Hq, d];
    k_new, v_new [B, Hkv, d]; k_cache, v_cache [B, L_max, Hkv, d]; cache_len int32 [B]."""
    B, L_max, Hkv, d = k_cache.shape
    Hq = q_new.shape[1]
    for t, nm, shp in ((q_new, "q_new", (B, Hq, d)), (qc_new, "qc_new", (B, Hq, d)),
                       (k_new, "k_new", (B, Hkv, d)), (v_new, "v_new", (B, Hkv, d)),
                       (k_cache, "k_cache", (B, L_max, Hkv, d)), (v_cache, "v_cache", (B, L_max, Hkv, d))):
        if t.dtype != torch.bfloat16 or not t.is_cuda or tuple(t.shape) != shp or not t.is_contiguous():
            raise OrthrosError(f"{nm} must be a contiguous bf16 CUDA tensor {shp}")
    if cache_len.dtype != torch.int32 or tuple(cache_len.shape) != (B,) or not cache_len.is_cuda:
        raise OrthrosError("cache_len must be an int32 CUDA tensor [B]")
    for t, nm in ((alpha, "alpha"), (beta, "beta"), (alpha_c, "alpha_c"), (beta_c, "beta_c")):
        _vec(t, nm, Hq, d)
    if o is None:
        o = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=k_cache.device)
    if oc is None:
        oc = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=k_cache.device)
    if workspace is None:
        workspace = decode_workspace(B, L_max, Hq, Hkv, d, k_cache.device)
    with torch.cuda.device(k_cache.device):
        st = lib().orthros_decode_step(_ptr(q_new), _ptr(qc_new), _ptr(k_new), _ptr(v_new),
                                       _ptr(k_cache), _ptr(v_cache), _ptr(cache_len), L_max,
                                       _ptr(alpha), _ptr(beta), _ptr(alpha_c), _ptr(beta_c),
                                       _ptr(o), _ptr(oc), B, Hq, Hkv, d, int(window), _scale(scale, d),
                                       _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _ptr(dev_err), _stream(k_cache.device))
    _check(st, "orthros_decode_step")
    return o, oc


_CODES = {torch.float8_e4m3fn: 0, torch.int8: 1}  # ORTHROS_KV_E4M3, ORTHROS_KV_INT8

# The calls below are made once a token and layer, so what they cost on the host counts: a
# tensor is checked and its address taken in one go, with as few attribute reads as will do,
# and addresses go to ctypes as plain integers.


def _refuse(t, name: str, what: str):
    raise OrthrosError(f"{name} must be a {what} on the call's device (got {tuple(t.shape)}, {t.dtype}, {t.device})")


def _dense(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on device `dev`."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _refuse(t, name, f"contiguous {dtype} CUDA tensor {tuple(shape)}")
    return t.data_ptr()


def _rows(t, name: str, shape, dev: int):
    """Address and batch stride of a bf16 tensor [B, T, H, d] whose [T, H, d] part is dense."""
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, f"bf16 CUDA tensor {tuple(shape)}")
    return t.data_ptr(), 0 if t.is_contiguous() else _bf16_rows(t, name)


def _optional(t, name: str, dtype, shape, dev: int):
    return None if t is None else _dense(t, name, dtype, shape, dev)


def _space(t, dev: int) -> int:
    """Address of a workspace on device `dev`."""
    if t.get_device() != dev or not t.is_contiguous():
        _refuse(t, "workspace", "contiguous CUDA tensor")
    return t.data_ptr()


def _word(t, dev: int):
    """Address of an error word on device `dev` (or None)."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() < 1 or t.get_device() != dev:
        _refuse(t, "dev_err", "int32 CUDA tensor")
    return t.data_ptr()


def _invoke(name: str, dev: int, *args) -> None:
    """Call an entry point on device `dev` and its current stream (the last argument of each)."""
    fn = getattr(_lib or lib(), name)
    if torch._C._cuda_getDevice() == dev:  # CUDA is initialised: there are tensors on it
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != 0:
        _check(st, name)


def _cache_q8(k8, v8, k_exp, v_exp):
    """Check the four tensors of an 8-bit cache; return ((B, L_max, Hkv, d, code), device, addresses)."""
    code, dev = _CODES.get(k8.dtype), k8.get_device()
    if code is None or k8.dim() != 4 or dev < 0:
        _refuse(k8, "k8", "contiguous float8_e4m3fn or int8 CUDA tensor [B, L_max, Hkv, d]")
    B, L_max, Hkv, d = shape = k8.shape
    exps = (B, Hkv, L_max)
    a = (_dense(k8, "k8", k8.dtype, shape, dev), _dense(v8, "v8", k8.dtype, shape, dev),
         _dense(k_exp, "k_exp", torch.int8, exps, dev), _dense(v_exp, "v_exp", torch.int8, exps, dev))
    return (B, L_max, Hkv, d, code), dev, a


def kv_cache_q8(B, L_max, Hkv, d, device, dtype=torch.float8_e4m3fn):
    """An empty 8-bit cache (k8, v8, k_exp, v_exp) of L_max rows, rounded up to a multiple of 16."""
    if dtype not in _CODES:
        raise OrthrosError("dtype must be torch.float8_e4m3fn or torch.int8")
    L_max = (L_max + 15) // 16 * 16
    codes = [torch.zeros((B, L_max, Hkv, d), dtype=torch.int8, device=device).view(dtype) for _ in range(2)]
    exps = [torch.zeros((B, Hkv, L_max), dtype=torch.int8, device=device) for _ in range(2)]
    return codes[0], codes[1], exps[0], exps[1]


def _kv_pair(k, v, B, Hkv, d, dev):
    """Check K and V rows [B, T, Hkv, d]; return (T, batch stride, addresses)."""
    shape = k.shape
    if k.dim() != 4 or shape[0] != B or shape[2] != Hkv or shape[3] != d:
        raise OrthrosError(f"k must be [B, T, Hkv, d] with B, Hkv, d = {B}, {Hkv}, {d}")
    ka, ks = _rows(k, "k", shape, dev)
    va, vs = _rows(v, "v", shape, dev)
    if vs != ks:
        raise OrthrosError("k and v must have the same shape and strides")
    return shape[1], ks, (ka, va)


def kv_quantize(k, v, k8, v8, k_exp, v_exp, start=None, rows=None, dev_err=None):
    """Write rows 0..rows[b]-1 (default all T) of k, v [B, T, Hkv, d] into the 8-bit cache at rows
    start[b].. (default 0): codes k8, v8 [B, L_max, Hkv, d] (float8_e4m3fn or int8) and exponents
    k_exp, v_exp int8 [B, Hkv, L_max]; a row stands for code * 2^exponent."""
    (B, L_max, Hkv, d, code), dev, cache = _cache_q8(k8, v8, k_exp, v_exp)
    T, ks, kv = _kv_pair(k, v, B, Hkv, d, dev)
    _invoke("orthros_kv_quantize", dev, *kv, _optional(start, "start", torch.int32, (B,), dev),
            _optional(rows, "rows", torch.int32, (B,), dev), *cache, B, T, Hkv, d, L_max, code, ks,
            _word(dev_err, dev))


def kv_dequantize(k8, v8, k_exp, v_exp, k, v, start=None, rows=None, dev_err=None):
    """Read cache rows start[b].. (default 0) back as bf16 into rows 0..rows[b]-1 (default all T) of
    k, v [B, T, Hkv, d]; rows behind them are left as they are.  Returns (k, v)."""
    (B, L_max, Hkv, d, code), dev, cache = _cache_q8(k8, v8, k_exp, v_exp)
    T, ks, kv = _kv_pair(k, v, B, Hkv, d, dev)
    _invoke("orthros_kv_dequantize", dev, *cache, _optional(start, "start", torch.int32, (B,), dev),
            _optional(rows, "rows", torch.int32, (B,), dev), *kv, B, T, Hkv, d, L_max, code, ks,
            _word(dev_err, dev))
    return k, v


def decode_q8_workspace_size(B, L_max, Hq, Hkv, d) -> int:
    return int(lib().orthros_decode_q8_workspace_size(B, L_max, Hq, Hkv, d))


def decode_q8_workspace(B, L_max, Hq, Hkv, d, device) -> torch.Tensor:
    """A zero-filled workspace for decode_step_q8 (reusable step after step)."""
    return torch.zeros(max(decode_q8_workspace_size(B, L_max, Hq, Hkv, d), 256), dtype=torch.uint8, device=device)


def _decode_args(q_new, qc_new, k_new, v_new, cache_len, alpha, beta, alpha_c, beta_c, o, oc, B, Hkv, d, dev):
    """Check what the decode steps share; return (o, oc, Hq, addresses of the new token's tensors, of
    cache_len, and of the vectors and outputs)."""
    Hq = q_new.shape[1]
    rows, new, vec, bf16, f32 = (B, Hq, d), (B, Hkv, d), (Hq, d), torch.bfloat16, torch.float32
    token = (_dense(q_new, "q_new", bf16, rows, dev), _dense(qc_new, "qc_new", bf16, rows, dev),
             _dense(k_new, "k_new", bf16, new, dev), _dense(v_new, "v_new", bf16, new, dev))
    o = torch.empty_like(q_new) if o is None else o
    oc = torch.empty_like(q_new) if oc is None else oc
    rest = (_dense(alpha, "alpha", f32, vec, dev), _dense(beta, "beta", f32, vec, dev),
            _dense(alpha_c, "alpha_c", f32, vec, dev), _dense(beta_c, "beta_c", f32, vec, dev),
            _dense(o, "o", bf16, rows, dev), _dense(oc, "oc", bf16, rows, dev))
    return o, oc, Hq, token, _dense(cache_len, "cache_len", torch.int32, (B,), dev), rest


def decode_step_q8(q_new, qc_new, k_new, v_new, k8, v8, k_exp, v_exp, cache_len, alpha, beta, alpha_c, beta_c,
                   window: int = 128, scale=None, o=None, oc=None, workspace=None, dev_err=None):
    """decode_step over an 8-bit cache (k8, v8 [B, L_max, Hkv, d] float8_e4m3fn or int8; k_exp, v_exp
    int8 [B, Hkv, L_max]): the new row is written as codes and both streams attend over the rows'
    values.  Returns (o, oc)."""
    (B, L_max, Hkv, d, code), dev, cache = _cache_q8(k8, v8, k_exp, v_exp)
    o, oc, Hq, token, lens, rest = _decode_args(q_new, qc_new, k_new, v_new, cache_len, alpha, beta, alpha_c, beta_c,
                                                o, oc, B, Hkv, d, dev)
    if workspace is None:
        workspace = decode_q8_workspace(B, L_max, Hq, Hkv, d, k8.device)
    _invoke("orthros_decode_step_q8", dev, *token, *cache, lens, L_max, code, *rest, B, Hq, Hkv, d, int(window),
            _scale(scale, d), _space(workspace, dev), workspace.nbytes, _word(dev_err, dev))
    return o, oc


def _prefix_rows(k_prefix, v_prefix, Hkv, d, dev):
    """Check the shared prefix [P, Hkv, d]; return (P, addresses)."""
    shape = (k_prefix.shape[0], Hkv, d)
    return shape[0], (_dense(k_prefix, "k_prefix", torch.bfloat16, shape, dev),
                      _dense(v_prefix, "v_prefix", torch.bfloat16, shape, dev))


def decode_prefix_workspace_size(B, P, L_max, Hq, Hkv, d) -> int:
    return int(lib().orthros_decode_prefix_workspace_size(B, P, L_max, Hq, Hkv, d))


def decode_prefix_workspace(B, P, L_max, Hq, Hkv, d, device) -> torch.Tensor:
    """A zero-filled workspace for decode_step_prefix (reusable step after step)."""
    return torch.zeros(max(decode_prefix_workspace_size(B, P, L_max, Hq, Hkv, d), 256), dtype=torch.uint8,
                       device=device)


def decode_step_prefix(q_new, qc_new, k_new, v_new, k_prefix, v_prefix, k_cache, v_cache, cache_len, alpha, beta,
                       alpha_c, beta_c, window: int = 128, scale=None, o=None, oc=None, workspace=None, dev_err=None):
    """decode_step for a batch that shares the prompt prefix k_prefix, v_prefix [P, Hkv, d]: sequence
    b's rows are the prefix and then its own cache_len[b] rows of k_cache, v_cache
    [B, L_max, Hkv, d].  Returns (o, oc)."""
    B, L_max, Hkv, d = shape = k_cache.shape
    dev = k_cache.get_device()
    if dev < 0:
        _refuse(k_cache, "k_cache", "contiguous bf16 CUDA tensor [B, L_max, Hkv, d]")
    cache = (_dense(k_cache, "k_cache", torch.bfloat16, shape, dev), _dense(v_cache, "v_cache", torch.bfloat16, shape, dev))
    P, prefix = _prefix_rows(k_prefix, v_prefix, Hkv, d, dev)
    o, oc, Hq, token, lens, rest = _decode_args(q_new, qc_new, k_new, v_new, cache_len, alpha, beta, alpha_c, beta_c,
                                                o, oc, B, Hkv, d, dev)
    if workspace is None:
        workspace = decode_prefix_workspace(B, P, L_max, Hq, Hkv, d, k_cache.device)
    _invoke("orthros_decode_step_prefix", dev, *token, *prefix, P, *cache, lens, L_max, *rest, B, Hq, Hkv, d,
            int(window), _scale(scale, d), _space(workspace, dev), workspace.nbytes,
            _word(dev_err, dev))
    return o, oc


def xattn_prefix_workspace_size(B, T_out, P, T_kv, Hq, Hkv, d) -> int:
    return int(lib().orthros_xattn_prefix_workspace_size(B, T_out, P, T_kv, Hq, Hkv, d))


def xattn_prefix_fwd(qc_raw, pos, k_prefix, v_prefix, k, v, alpha_c, beta_c, scale=None, out=None, workspace=None,
                     dev_err=None):
    """xattn_fwd for a batch that shares the prompt prefix k_prefix, v_prefix [P, Hkv, d]: copy i of
    sequence b attends over the prefix and its sequence's own rows 0..pos[b, i] of k, v
    [B, T_kv, Hkv, d].  qc_raw [B, T_out, Hq, d]; pos int32 [B, T_out]."""
    B, T_kv, Hkv, d = k.shape
    dev = k.get_device()
    if dev < 0:
        _refuse(k, "k", "bf16 CUDA tensor [B, T_kv, Hkv, d]")
    _, T_out, Hq, _ = qc_raw.shape
    shape = (B, T_out, Hq, d)
    _, ks, own = _kv_pair(k, v, B, Hkv, d, dev)
    qa, qs = _rows(qc_raw, "qc_raw", shape, dev)
    P, prefix = _prefix_rows(k_prefix, v_prefix, Hkv, d, dev)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=k.device)
    oa, os_ = _rows(out, "out", shape, dev)
    if workspace is None:
        workspace = torch.empty(max(xattn_prefix_workspace_size(B, T_out, P, T_kv, Hq, Hkv, d), 256),
                                dtype=torch.uint8, device=k.device)
    _invoke("orthros_xattn_prefix_fwd", dev, qa, _dense(pos, "pos", torch.int32, (B, T_out), dev), *prefix, P, *own,
            _dense(alpha_c, "alpha_c", torch.float32, (Hq, d), dev),
            _dense(beta_c, "beta_c", torch.float32, (Hq, d), dev), oa, B, T_out, T_kv, Hq, Hkv, d, _scale(scale, d),
            qs, ks, os_, _space(workspace, dev), workspace.nbytes, _word(dev_err, dev))
    return out


def swa_sink_fwd(q_raw, k, v, alpha, beta, sinks: int, window: int = 128, scale=None, out=None, lse=None,
                 row_begin: int = 0, row_end=None, dev_err=None):
    """swa_fwd with attention sinks: row t attends over keys j <= t with j > t - window or j < sinks
    (0 <= sinks <= 32).  Only rows row_begin..row_end-1 (default all T) are computed, by swa_fwd_rows'
    rules.  With lse (fp32 [B, T, Hq], or True for a fresh one) each row's log-sum-exp is written too,
    for swa_sink_bwd, and (out, lse) is returned."""
    B, T, Hkv, d = kv_shape = k.shape
    dev = k.get_device()
    if dev < 0:
        _refuse(k, "k", "bf16 CUDA tensor [B, T, Hkv, d]")
    ka, ks = _rows(k, "k", kv_shape, dev)
    va, vs = _rows(v, "v", kv_shape, dev)
    if vs != ks:
        raise OrthrosError("k and v must have the same shape and strides")
    q_shape = q_raw.shape
    if len(q_shape) != 4 or q_shape[0] != B or q_shape[1] < T or q_shape[3] != d:
        raise OrthrosError("q_raw shape does not match k")
    Tq, Hq = q_shape[1], q_shape[2]
    qa, qs = _rows(q_raw, "q_raw", q_shape, dev)
    if qs == 0:  # dense, but it may hold appended copies
        qs = Tq * Hq * d
    shape = (B, T, Hq, d)
    if out is None:
        out = torch.empty_like(q_raw) if Tq == T and q_raw.is_contiguous() else torch.empty(
            shape, dtype=torch.bfloat16, device=k.device)
    oa, os_ = _rows(out, "out", shape, dev)
    if lse is True:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=k.device)
    _invoke("orthros_swa_sink_fwd", dev, qa, ka, va, _dense(alpha, "alpha", torch.float32, (Hq, d), dev),
            _dense(beta, "beta", torch.float32, (Hq, d), dev), oa,
            _optional(lse, "lse", torch.float32, (B, T, Hq), dev), B, T, Hq, Hkv, d, int(window), int(sinks),
            _scale(scale, d), qs, ks, os_, int(row_begin), T if row_end is None else int(row_end), _word(dev_err, dev))
    return out if lse is None else (out, lse)


def swa_sink_bwd_workspace_size(B, T, Hq, Hkv, d) -> int:
    return int(lib().orthros_swa_sink_bwd_workspace_size(B, T, Hq, Hkv, d))


def swa_sink_bwd(q_raw, k, v, alpha, beta, o, dO, lse, sinks: int, window: int = 128, scale=None, workspace=None,
                 dev_err=None):
    """Gradient of swa_sink_fwd: returns fp32 (dq_raw, dk, dv, dalpha, dbeta) for the output gradient dO, given the
    forward's inputs, output o and log-sum-exp lse (fp32 [B, T, Hq]).  q_raw, o, dO [B, T, Hq, d] and k, v
    [B, T, Hkv, d], all dense bf16; alpha, beta [Hq, d] fp32.  xattn_bwd adds the copies' share to dk, dv."""
    B, T, Hkv, d = kv = k.shape
    dev = k.get_device()
    if dev < 0:
        _refuse(k, "k", "contiguous bf16 CUDA tensor [B, T, Hkv, d]")
    Hq = q_raw.shape[2]
    rows, vec, bf16, f32 = (B, T, Hq, d), (Hq, d), torch.bfloat16, torch.float32
    args = (_dense(q_raw, "q_raw", bf16, rows, dev), _dense(k, "k", bf16, kv, dev), _dense(v, "v", bf16, kv, dev),
            _dense(alpha, "alpha", f32, vec, dev), _dense(beta, "beta", f32, vec, dev), _dense(o, "o", bf16, rows, dev),
            _dense(dO, "dO", bf16, rows, dev), _dense(lse, "lse", f32, (B, T, Hq), dev))
    out = [torch.empty(shape, dtype=f32, device=k.device) for shape in (rows, kv, kv, vec, vec)]
    if workspace is None:
        workspace = torch.empty(max(swa_sink_bwd_workspace_size(B, T, Hq, Hkv, d), 256), dtype=torch.uint8,
                                device=k.device)
    _invoke("orthros_swa_sink_bwd", dev, *args, *[t.data_ptr() for t in out], B, T, Hq, Hkv, d, int(window), int(sinks),
            _scale(scale, d), _space(workspace, dev), workspace.nbytes, _word(dev_err, dev))
    return tuple(out)


def decode_tree_workspace_size(B, N, L_max, Hq, Hkv, d) -> int:
    return int(lib().orthros_decode_tree_workspace_size(B, N, L_max, Hq, Hkv, d))


def decode_tree(q_new, qc_new, k_new, v_new, parent, k_cache, v_cache, cache_len, alpha, beta, alpha_c, beta_c,
                window: int = 128, sinks: int = 0, nodes=None, scale=None, o=None, oc=None, workspace=None,
                dev_err=None):
    """Both streams of a tree of N <= 64 drafted tokens over a cache; nothing is appended (decode_tree_accept).
    Node i of sequence b hangs below node parent[b, i] < i, or below the last cached row (-1).  Its copy
    qc_new[b, i] attends over cache rows 0..cache_len[b]-1 and the rows of its path (ancestors and itself) in
    k_new, v_new; its base token q_new[b, i] over those of them in its window or among the first `sinks`
    positions.  q_new, qc_new [B, N, Hq, d]; k_new, v_new [B, N, Hkv, d]; parent int32 [B, N]; k_cache, v_cache
    [B, L_max, Hkv, d]; cache_len int32 [B]; nodes int32 [B]: nodes of each tree (default N; rows of o, oc behind
    them are left as they are).  Returns (o, oc)."""
    B, L_max, Hkv, d = shape = k_cache.shape
    dev = k_cache.get_device()
    if dev < 0 or q_new.dim() != 4:
        _refuse(q_new if dev >= 0 else k_cache, "q_new and k_cache", "contiguous bf16 CUDA tensor of four dimensions")
    _, N, Hq, _ = q_new.shape
    rows, new, vec, bf16, f32, i32 = (B, N, Hq, d), (B, N, Hkv, d), (Hq, d), torch.bfloat16, torch.float32, torch.int32
    o = torch.empty_like(q_new) if o is None else o
    oc = torch.empty_like(q_new) if oc is None else oc
    if workspace is None:
        workspace = torch.empty(max(decode_tree_workspace_size(B, N, L_max, Hq, Hkv, d), 256), dtype=torch.uint8,
                                device=k_cache.device)
    _invoke("orthros_decode_tree", dev, _dense(q_new, "q_new", bf16, rows, dev), _dense(qc_new, "qc_new", bf16, rows, dev),
            _dense(k_new, "k_new", bf16, new, dev), _dense(v_new, "v_new", bf16, new, dev),
            _dense(parent, "parent", i32, (B, N), dev), _optional(nodes, "nodes", i32, (B,), dev),
            _dense(k_cache, "k_cache", bf16, shape, dev), _dense(v_cache, "v_cache", bf16, shape, dev),
            _dense(cache_len, "cache_len", i32, (B,), dev), L_max, _dense(alpha, "alpha", f32, vec, dev),
            _dense(beta, "beta", f32, vec, dev), _dense(alpha_c, "alpha_c", f32, vec, dev),
            _dense(beta_c, "beta_c", f32, vec, dev), _dense(o, "o", bf16, rows, dev), _dense(oc, "oc", bf16, rows, dev),
            B, N, Hq, Hkv, d, int(window), int(sinks), _scale(scale, d), _space(workspace, dev), workspace.nbytes,
            _word(dev_err, dev))
    return o, oc


def decode_tree_accept(k_new, v_new, parent, node, k_cache, v_cache, cache_len, path=None, dev_err=None, nodes=None):
    """Append what the check of a drafted tree accepted: the rows of k_new, v_new [B, N, Hkv, d] on the path to
    node[b] (int32 [B]; -1: none) go to cache rows cache_len[b].., and cache_len[b] grows by their number.  nodes as
    given to decode_tree: node[b] is one of its tree's, 0..nodes[b]-1 (default N), or -1.
    Returns path, int32 [B, N]: the path's nodes in order, -1 behind the last."""
    B, L_max, Hkv, d = shape = k_cache.shape
    dev = k_cache.get_device()
    if dev < 0 or k_new.dim() != 4:
        _refuse(k_new if dev >= 0 else k_cache, "k_new and k_cache", "contiguous bf16 CUDA tensor of four dimensions")
    N = k_new.shape[1]
    new, bf16, i32 = (B, N, Hkv, d), torch.bfloat16, torch.int32
    if path is None:
        path = torch.empty((B, N), dtype=i32, device=k_cache.device)
    _invoke("orthros_decode_tree_accept_nodes", dev, _dense(k_new, "k_new", bf16, new, dev),
            _dense(v_new, "v_new", bf16, new, dev), _dense(parent, "parent", i32, (B, N), dev),
            _optional(nodes, "nodes", i32, (B,), dev), _dense(node, "node", i32, (B,), dev),
            _dense(k_cache, "k_cache", bf16, shape, dev),
            _dense(v_cache, "v_cache", bf16, shape, dev), _dense(cache_len, "cache_len", i32, (B,), dev), L_max,
            _dense(path, "path", i32, (B, N), dev), B, N, Hkv, d, _word(dev_err, dev))
    return path
