"""Python binding of libckda -- the GB300 (sm_103a) Complex KDA recurrence.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libckda.so (csrc/), called through its C ABI (include/ckda.h).
PyTorch supplies device memory and streams.  There is no CPU or PyTorch
fallback: if the library is missing or fails to load, every call raises.

    o, hT = fwd(q, k, v, alpha, beta, h0=None, cu_seqlens=None, scale=1.0)
    o = decode_step(q, k, v, alpha, beta, state)      # state updated in place

Next to the recurrence are linear attention with a scalar decay per head
(linear_fwd, linear_bwd, linear_decode_step) and layer norm (layernorm_fwd,
layernorm_bwd), and the parts of a state space block: the short causal
convolution (conv_fwd, conv_bwd, conv_decode_step), the selective scan
(scan_fwd, scan_bwd, scan_decode_step) and RMS norm with a residual's addition
and outputs in 8 bits (rmsnorm_fwd, rmsnorm_fwd8, rmsnorm_bwd).

Shapes follow the C ABI: q, k, alpha [B, H, T, dk]; v [B, H, T, dv];
beta [B, H, T]; h0 / hT fp32 [N, H, dk, dv] with N = B, or the number of
packed sequences when cu_seqlens (int32 [N + 1], B == 1) is given.

Calls run on the current stream of the tensors' device, or on `stream`.  With a
stream of its own, a call takes its memory there too; that the stream sees its
inputs, and the caller's its results, is the caller's part (wait_stream), as it
is for torch's own calls under torch.cuda.stream.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

__all__ = ["fwd", "fwd_host", "fwd_split", "decode_step", "decode_step_raw", "prep", "bwd",
           "bwd_workspace_bytes", "fwd_status", "workspace_bytes", "split_segments",
           "split_workspace_bytes", "host_scratch_bytes", "selftest_timeout", "lib",
           "library_path", "CkdaError", "STATUS", "recurrence", "prepare", "linear_fwd",
           "linear_bwd", "linear_decode_step", "linear_attention", "layernorm_fwd",
           "layernorm_bwd", "layer_norm", "conv_fwd", "conv_bwd", "conv_decode_step",
           "short_conv", "scan_fwd", "scan_bwd", "scan_decode_step", "selective_scan",
           "rmsnorm_fwd", "rmsnorm_fwd8", "rmsnorm_bwd", "rms_norm"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libckda.so")
_lock = threading.Lock()
_lib = None

STATUS = {0: "CKDA_OK", 1: "CKDA_ERR_INVALID_ARG", 2: "CKDA_ERR_UNSUPPORTED",
          3: "CKDA_ERR_CUDA", 4: "CKDA_ERR_TIMEOUT", 5: "CKDA_ERR_WORKSPACE",
          6: "CKDA_ERR_RANGE"}
_F32, _BF16 = 0, 1


class CkdaError(RuntimeError):
    def __init__(self, code, where):
        self.code = int(code)
        super().__init__(f"{where}: {STATUS.get(self.code, self.code)}")


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded libckda (ctypes.CDLL).  Raises if the library is not built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise ImportError(
                    f"libckda.so is not built ({_LIB_PATH}); run "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(_LIB_PATH)
            vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
            L.ckda_version.restype = i32
            L.ckda_version.argtypes = []
            L.ckda_status_string.restype = ctypes.c_char_p
            L.ckda_status_string.argtypes = [i32]
            L.ckda_fwd_workspace_bytes.restype = sz
            L.ckda_fwd_workspace_bytes.argtypes = [i32, i32]
            L.ckda_fwd.restype = i32
            L.ckda_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32,
                                   i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp]
            L.ckda_fwd_status.restype = i32
            L.ckda_fwd_status.argtypes = [vp, vp]
            L.ckda_decode_step.restype = i32
            L.ckda_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp,
                                           i32, i32, i32, i32, i32, f32, vp]
            L.ckda_selftest_timeout.restype = i32
            L.ckda_selftest_timeout.argtypes = [vp, sz, ctypes.c_uint, vp]
            L.ckda_fwd_host_scratch_bytes.restype = sz
            L.ckda_fwd_host_scratch_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
            L.ckda_decode_step_raw.restype = i32
            L.ckda_decode_step_raw.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                               i32, f32, i32, f32, vp]
            L.ckda_bwd_workspace_bytes.restype = sz
            L.ckda_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
            L.ckda_bwd.restype = i32
            L.ckda_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   i32, i32, i32, i32, i32, i32, i32, f32, vp, sz, vp]
            L.ckda_prep.restype = i32
            L.ckda_prep.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_longlong, i32, i32,
                                    i32, f32, vp]
            L.ckda_fwd_split_varlen_seg_len.restype = i32
            L.ckda_fwd_split_varlen_seg_len.argtypes = [i32] * 7
            L.ckda_fwd_split_varlen_workspace_bytes.restype = sz
            L.ckda_fwd_split_varlen_workspace_bytes.argtypes = [i32] * 5
            L.ckda_fwd_split_varlen.restype = i32
            L.ckda_fwd_split_varlen.argtypes = [vp] * 9 + [i32] * 6 + [f32, i32, vp, sz, vp]
            L.ckda_fwd_raw.restype = i32
            L.ckda_fwd_raw.argtypes = [vp] * 9 + [i32] * 7 + [f32, i32, f32, vp, sz, vp]
            L.ckda_prep_bwd.restype = i32
            L.ckda_prep_bwd.argtypes = [vp] * 12 + [ctypes.c_longlong, i32, i32, i32, f32, vp]
            L.ckda_fwd_host.restype = i32
            L.ckda_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                        i32, f32, i32, vp, sz, vp]
            L.ckda_fwd_split_segments.restype = i32
            L.ckda_fwd_split_segments.argtypes = [i32, i32, i32, i32, i32, i32, i32]
            L.ckda_fwd_split_workspace_bytes.restype = sz
            L.ckda_fwd_split_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
            L.ckda_fwd_split.restype = i32
            L.ckda_fwd_split.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                         i32, f32, i32, vp, sz, vp]
            lin = [vp, vp, vp, vp, i32, vp]
            for n, fn in ((7, L.ckda_linear_fwd_workspace_bytes),
                          (7, L.ckda_linear_fwd_aligned_workspace_bytes),
                          (8, L.ckda_linear_bwd_workspace_bytes),
                          (8, L.ckda_linear_bwd_aligned_workspace_bytes)):
                fn.restype, fn.argtypes = sz, [i32] * n
            L.ckda_linear_fwd.restype = i32
            L.ckda_linear_fwd.argtypes = lin + [vp] * 3 + [i32] * 8 + [f32, vp, sz, vp]
            L.ckda_linear_bwd.restype = i32
            L.ckda_linear_bwd.argtypes = lin + [vp] * 8 + [i32] * 8 + [f32, vp, sz, vp]
            L.ckda_linear_decode_step.restype = i32
            L.ckda_linear_decode_step.argtypes = [vp] * 4 + [i32, vp, vp] + [i32] * 6 + [f32, vp]
            L.ckda_layernorm_fwd.restype = i32
            L.ckda_layernorm_fwd.argtypes = [vp] * 6 + [ctypes.c_longlong, i32, i32, i32, f32, vp]
            L.ckda_layernorm_bwd_workspace_bytes.restype = sz
            L.ckda_layernorm_bwd_workspace_bytes.argtypes = [ctypes.c_longlong, i32]
            L.ckda_layernorm_bwd.restype = i32
            L.ckda_layernorm_bwd.argtypes = [vp] * 8 + [ctypes.c_longlong, i32, i32, i32, vp, sz,
                                                        vp]
            i64 = ctypes.c_longlong
            for fn in (L.ckda_conv_fwd, L.ckda_conv_fwd_filled):
                fn.restype = i32
                fn.argtypes = [vp] * 7 + [i32] * 5 + [i64] + [i32] * 3 + [vp]
            L.ckda_conv_bwd_workspace_bytes.restype = sz
            L.ckda_conv_bwd_workspace_bytes.argtypes = [i32] * 4
            L.ckda_conv_bwd.restype = i32
            L.ckda_conv_bwd.argtypes = [vp] * 11 + [i32] * 5 + [i64] + [i32] * 3 + [vp, sz, vp]
            L.ckda_conv_decode_step.restype = i32
            L.ckda_conv_decode_step.argtypes = [vp] * 5 + [i32] * 3 + [i64] + [i32] * 3 + [vp]
            for fn in (L.ckda_scan_fwd_workspace_bytes, L.ckda_scan_bwd_workspace_bytes):
                fn.restype, fn.argtypes = sz, [i32] * 5
            for fn in (L.ckda_scan_fwd, L.ckda_scan_fwd_filled):
                fn.restype = i32
                fn.argtypes = [vp] * 12 + [i32] * 6 + [i64] * 5 + [i32] * 2 + [vp, sz, vp]
            L.ckda_scan_bwd.restype = i32
            L.ckda_scan_bwd.argtypes = [vp] * 21 + [i32] * 6 + [i64] * 5 + [i32] * 2 + [vp, sz, vp]
            L.ckda_scan_decode_step.restype = i32
            L.ckda_scan_decode_step.argtypes = [vp] * 10 + [i32] * 4 + [i64] * 5 + [i32] * 2 + [vp]
            L.ckda_rmsnorm_fwd.restype = i32
            L.ckda_rmsnorm_fwd.argtypes = [vp] * 6 + [i64] + [i32] * 3 + [f32, vp]
            L.ckda_rmsnorm_fwd8.restype = i32
            L.ckda_rmsnorm_fwd8.argtypes = [vp] * 7 + [i64] + [i32] * 4 + [f32, vp]
            L.ckda_rmsnorm_bwd_workspace_bytes.restype = sz
            L.ckda_rmsnorm_bwd_workspace_bytes.argtypes = [i64, i32]
            L.ckda_rmsnorm_bwd.restype = i32
            L.ckda_rmsnorm_bwd.argtypes = [vp] * 7 + [i64] + [i32] * 3 + [vp, sz, vp]
            _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device):
    if device.type != "cuda":
        raise ValueError(f"tensors on {device}, expected CUDA")
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _on_stream(call, args):
    """call(**args) where args["stream"] is given: with that stream current, so that what the
    call allocates is the stream's memory, which goes to another use behind the call's kernels
    and not beside them.  The results may be used, and freed, on the caller's stream too."""
    stream = args.pop("stream")
    tensors = [t for t in args.values() if isinstance(t, torch.Tensor)]
    for t in tensors:
        if t.is_cuda and t.device != stream.device:
            raise ValueError(f"stream: on {stream.device}, expected {t.device}")
    here = torch.cuda.current_stream(stream.device)
    if stream == here:
        return call(**args)
    with torch.cuda.stream(stream):
        out = call(**args)
    given = {id(t) for a in args.values() for t in (a if isinstance(a, (tuple, list)) else (a,))}
    for t in out if isinstance(out, tuple) else (out,):
        if isinstance(t, torch.Tensor) and t.is_cuda and id(t) not in given:
            t.record_stream(here)
    return out


def _io_dtype(t):
    if t.dtype == torch.bfloat16:
        return _BF16
    if t.dtype == torch.float32:
        return _F32
    raise TypeError(f"unsupported I/O dtype {t.dtype} (bf16 or fp32)")


def _check(t, name, dtype, shape, device):
    if t.dtype == dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _given(t, device, name="workspace"):
    """Bytes of scratch memory that the caller gave: on the tensors' device, in one run."""
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.numel() * t.element_size()


def workspace_bytes(num_seqs: int, H: int) -> int:
    return int(lib().ckda_fwd_workspace_bytes(int(num_seqs), int(H)))


def new_workspace(num_seqs, H, device):
    n = workspace_bytes(num_seqs, H)
    return torch.empty(n, dtype=torch.uint8, device=device)


def fwd_raw(q_raw, k_raw, v, a_raw, b_raw, h0=None, cu_seqlens=None, scale=1.0,
            normalize_q=True, norm_eps=1e-6, store_final_state=True, o=None, hT=None,
            workspace=None, stream=None):
    """ckda_fwd_raw: the forward on raw q, k and gate logits a, b, with the
    input preparation of `prep` applied inside the kernel.  Returns (o, hT or
    None)."""
    return fwd(q_raw, k_raw, v, a_raw, b_raw, h0, cu_seqlens, scale, 0, store_final_state, o,
               hT, workspace, stream, _raw=(bool(normalize_q), float(norm_eps)))


def fwd(q, k, v, alpha, beta, h0=None, cu_seqlens=None, scale=1.0, chunk_size=0,
        store_final_state=True, o=None, hT=None, workspace=None, stream=None, _raw=None):
    """Forward over [B, H, T, d] (or packed) inputs.  Returns (o, hT or None)."""
    if stream is not None:
        return _on_stream(fwd, locals())
    L = lib()
    device = q.device
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _io_dtype(q)
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)),
                         ("alpha", alpha, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("beta", beta, (B, H, T))):
        _check(t, name, dt, shp, device)
    N = B
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), device)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv), device)
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=dt, device=device)
    else:
        _check(o, "o", dt, (B, H, T, dv), device)
    if store_final_state and hT is None:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=device)
    if hT is not None:
        _check(hT, "hT", torch.float32, (N, H, dk, dv), device)
    nseq_ws = N if cu_seqlens is not None else 0
    if workspace is None:
        workspace = new_workspace(nseq_ws, H, device)
    nseq = int(N if cu_seqlens is not None else 0)
    if _raw is None:
        rc = L.ckda_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(o),
                        _ptr(hT), _ptr(cu_seqlens), nseq, B, H, T, dk, dv, _io_dtype(q),
                        float(scale), int(chunk_size), _ptr(workspace), _given(workspace, device),
                        _stream_handle(None, device))
    else:
        rc = L.ckda_fwd_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(o),
                            _ptr(hT), _ptr(cu_seqlens), nseq, B, H, T, dk, dv, _io_dtype(q),
                            float(scale), int(_raw[0]), float(_raw[1]), _ptr(workspace),
                            _given(workspace, device), _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_fwd" if _raw is None else "ckda_fwd_raw")
    fwd.last_workspace = workspace
    fwd_raw.last_workspace = workspace
    return o, hT


def split_segments(B, H, T, dk, dv, dtype=torch.bfloat16, num_sms=0) -> int:
    """Segment count ckda_fwd_split picks for `segments=0` (num_sms = 0: the
    current device's SM count)."""
    io = _BF16 if dtype == torch.bfloat16 else _F32
    return int(lib().ckda_fwd_split_segments(B, H, T, dk, dv, io, int(num_sms)))


def split_workspace_bytes(B, H, T, dk, dv, dtype=torch.bfloat16, segments=0) -> int:
    io = _BF16 if dtype == torch.bfloat16 else _F32
    return int(lib().ckda_fwd_split_workspace_bytes(B, H, T, dk, dv, io, int(segments)))


def fwd_split(q, k, v, alpha, beta, h0=None, scale=1.0, segments=0, store_final_state=True,
              o=None, hT=None, workspace=None, stream=None):
    """ckda_fwd_split: the dense forward with each sequence cut into segments
    run in parallel (two passes and a scan of the segment operators).
    Returns (o, hT or None)."""
    if stream is not None:
        return _on_stream(fwd_split, locals())
    L = lib()
    device = q.device
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    io = _io_dtype(q)
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)),
                         ("alpha", alpha, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("beta", beta, (B, H, T))):
        _check(t, name, dt, shp, device)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv), device)
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=dt, device=device)
    else:
        _check(o, "o", dt, (B, H, T, dv), device)
    if store_final_state and hT is None:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=device)
    if hT is not None:
        _check(hT, "hT", torch.float32, (B, H, dk, dv), device)
    if workspace is None:
        with torch.cuda.device(device):
            n = int(L.ckda_fwd_split_workspace_bytes(B, H, T, dk, dv, io, int(segments)))
        workspace = torch.empty(n, dtype=torch.uint8, device=device)
    with torch.cuda.device(device):
        rc = L.ckda_fwd_split(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0),
                              _ptr(o), _ptr(hT), B, H, T, dk, dv, io, float(scale),
                              int(segments), _ptr(workspace), _given(workspace, device),
                              _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_fwd_split")
    fwd_split.last_workspace = workspace
    return o, hT


def split_varlen_seg_len(num_seqs, H, T, dk, dv, dtype=torch.bfloat16, num_sms=0) -> int:
    """Segment length ckda_fwd_split_varlen picks for `seg_len=0`."""
    io = _BF16 if dtype == torch.bfloat16 else _F32
    return int(lib().ckda_fwd_split_varlen_seg_len(num_seqs, H, T, dk, dv, io, int(num_sms)))


def split_varlen_workspace_bytes(num_seqs, H, T, dk, seg_len) -> int:
    return int(lib().ckda_fwd_split_varlen_workspace_bytes(num_seqs, H, T, dk, int(seg_len)))


def fwd_split_varlen(q, k, v, alpha, beta, cu_seqlens, h0=None, scale=1.0, seg_len=0,
                     store_final_state=True, o=None, hT=None, workspace=None, stream=None):
    """ckda_fwd_split_varlen: the packed forward with every sequence longer
    than seg_len cut into segments run in parallel.  q, k, alpha, v are
    [1, H, T, d], beta [1, H, T], cu_seqlens int32 [N + 1] on the device.
    Returns (o, hT [N, H, dk, dv] or None)."""
    if stream is not None:
        return _on_stream(fwd_split_varlen, locals())
    L = lib()
    device = q.device
    B, H, T, dk = q.shape
    if B != 1:
        raise ValueError("fwd_split_varlen: packed input has B = 1")
    dv = v.shape[-1]
    dt = q.dtype
    io = _io_dtype(q)
    for name, t, shp in (("q", q, (1, H, T, dk)), ("k", k, (1, H, T, dk)),
                         ("alpha", alpha, (1, H, T, dk)), ("v", v, (1, H, T, dv)),
                         ("beta", beta, (1, H, T))):
        _check(t, name, dt, shp, device)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != device or cu_seqlens.dim() != 1:
        raise ValueError("fwd_split_varlen: cu_seqlens must be int32 [N + 1] on the device")
    N = cu_seqlens.numel() - 1
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv), device)
    if o is None:
        o = torch.empty((1, H, T, dv), dtype=dt, device=device)
    else:
        _check(o, "o", dt, (1, H, T, dv), device)
    if store_final_state and hT is None:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=device)
    if hT is not None:
        _check(hT, "hT", torch.float32, (N, H, dk, dv), device)
    with torch.cuda.device(device):
        if seg_len == 0:
            seg_len = int(L.ckda_fwd_split_varlen_seg_len(N, H, T, dk, dv, io, 0))
        if workspace is None:
            n = int(L.ckda_fwd_split_varlen_workspace_bytes(N, H, T, dk, int(seg_len)))
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
        rc = L.ckda_fwd_split_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0),
                                     _ptr(o), _ptr(hT), _ptr(cu_seqlens), N, H, T, dk, dv, io,
                                     float(scale), int(seg_len), _ptr(workspace),
                                     _given(workspace, device), _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_fwd_split_varlen")
    fwd_split_varlen.last_workspace = workspace
    return o, hT


def fwd_status(workspace, stream=None) -> int:
    """Device status of the most recent call on `workspace` (synchronises)."""
    return int(lib().ckda_fwd_status(_ptr(workspace), _stream_handle(stream, workspace.device)))


def host_scratch_bytes(B, H, T, dk, dv, dtype=torch.bfloat16, slice_tokens=0) -> int:
    io = _BF16 if dtype == torch.bfloat16 else _F32
    return int(lib().ckda_fwd_host_scratch_bytes(B, H, T, dk, dv, io, int(slice_tokens)))


def fwd_host(q, k, v, alpha, beta, h0=None, scale=1.0, slice_tokens=0, o=None, hT=None,
             store_final_state=True, scratch=None, stream=None, device=None):
    """ckda_fwd_host: the dense forward with every tensor in host memory (CPU
    tensors; pinned memory copies at full speed).  The copies of one slice of
    tokens overlap the computation of another.  Returns (o, hT or None) as CPU
    tensors; they are complete once `stream` is (this call does not wait)."""
    if stream is not None:
        return _on_stream(fwd_host, locals())
    L = lib()
    device = torch.device("cuda" if device is None else device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    io = _io_dtype(q)
    cpu = torch.device("cpu")
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)),
                         ("alpha", alpha, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("beta", beta, (B, H, T))):
        _check(t, name, dt, shp, cpu)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv), cpu)
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=dt).pin_memory()
    else:
        _check(o, "o", dt, (B, H, T, dv), cpu)
    if store_final_state and hT is None:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32).pin_memory()
    if hT is not None:
        _check(hT, "hT", torch.float32, (B, H, dk, dv), cpu)
    need = host_scratch_bytes(B, H, T, dk, dv, dt, slice_tokens)
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device=device)
    rc = L.ckda_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(o),
                         _ptr(hT), B, H, T, dk, dv, io, float(scale), int(slice_tokens),
                         _ptr(scratch), _given(scratch, device, "scratch"),
                         _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_fwd_host")
    fwd_host.last_scratch = scratch
    return o, hT


def decode_step(q, k, v, alpha, beta, state, scale=1.0, o=None, stream=None):
    """One token per (batch, head); `state` [B, H, dk, dv] fp32 is updated in place."""
    if stream is not None:
        return _on_stream(decode_step, locals())
    L = lib()
    device = q.device
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _io_dtype(q)
    for name, t, shp in (("q", q, (B, H, dk)), ("k", k, (B, H, dk)), ("alpha", alpha, (B, H, dk)),
                         ("v", v, (B, H, dv)), ("beta", beta, (B, H))):
        _check(t, name, dt, shp, device)
    _check(state, "state", torch.float32, (B, H, dk, dv), device)
    if o is None:
        o = torch.empty((B, H, dv), dtype=dt, device=device)
    else:
        _check(o, "o", dt, (B, H, dv), device)
    rc = L.ckda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state),
                            _ptr(o), B, H, dk, dv, _io_dtype(q), float(scale),
                            _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_decode_step")
    return o


def selftest_timeout(workspace, spin_limit=1000, stream=None) -> int:
    """Runs the bounded-wait self-test and returns the status it recorded."""
    L = lib()
    rc = L.ckda_selftest_timeout(_ptr(workspace), int(workspace.numel()), int(spin_limit),
                                 _stream_handle(stream, workspace.device))
    if rc != 0:
        raise CkdaError(rc, "ckda_selftest_timeout")
    return fwd_status(workspace, stream)


def fwd_noalloc(q, k, v, alpha, beta, h0=None, cu_seqlens=None, scale=1.0, chunk_size=0,
                o=None, hT=None, stream=None):
    """ckda_fwd_noalloc: the forward without a workspace, for callers that may
    not allocate device memory (its scratch is a fixed array inside libckda).
    o and hT may be passed in so that the call itself allocates nothing."""
    if stream is not None:
        return _on_stream(fwd_noalloc, locals())
    L = lib()
    fn = L.ckda_fwd_noalloc
    if fn.argtypes is None:
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        fn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32,
                       i32, i32, i32, i32, i32, i32, f32, i32, vp]
        fn.restype = i32
    device = q.device
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)),
                         ("alpha", alpha, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("beta", beta, (B, H, T))):
        _check(t, name, q.dtype, shp, device)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), device)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv), device)
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=q.dtype, device=device)
    else:
        _check(o, "o", q.dtype, (B, H, T, dv), device)
    if hT is None:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=device)
    else:
        _check(hT, "hT", torch.float32, (N, H, dk, dv), device)
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT),
            _ptr(cu_seqlens), int(N if cu_seqlens is not None else 0), B, H, T, dk, dv,
            _io_dtype(q), float(scale), int(chunk_size), _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_fwd_noalloc")
    return o, hT


def prep(k_raw, a_raw, b_raw, q_raw=None, normalize_q=True, norm_eps=1e-6, out=None,
         stream=None):
    """Fused input preparation (ckda_prep): unit-norm keys (and queries when
    normalize_q), alpha = s[e^-5 + (1 - e^-5)|tanh(a/2)|], beta = 2 sigmoid(b).

    k_raw, a_raw (and q_raw) are [..., dk]; b_raw is [...].  Returns
    (q or None, k, alpha, beta) in the input dtype.  `out` may give the four
    output tensors (q may be None); passing the inputs themselves works in place.
    """
    if stream is not None:
        return _on_stream(prep, locals())
    L = lib()
    device = k_raw.device
    dt = k_raw.dtype
    dk = k_raw.shape[-1]
    _check(a_raw, "a_raw", dt, tuple(k_raw.shape), device)
    _check(b_raw, "b_raw", dt, tuple(k_raw.shape[:-1]), device)
    if q_raw is not None:
        _check(q_raw, "q_raw", dt, tuple(k_raw.shape), device)
    _check(k_raw, "k_raw", dt, tuple(k_raw.shape), device)
    if out is None:
        q = None if q_raw is None else torch.empty_like(q_raw)
        k, alpha, beta = torch.empty_like(k_raw), torch.empty_like(a_raw), torch.empty_like(b_raw)
    else:
        q, k, alpha, beta = out
        for name, t, shp in (("k", k, k_raw.shape), ("alpha", alpha, k_raw.shape),
                             ("beta", beta, k_raw.shape[:-1])):
            _check(t, name, dt, tuple(shp), device)
        if (q is None) != (q_raw is None):
            raise ValueError("prep: q and q_raw must both be given or both be None")
        if q is not None:
            _check(q, "q", dt, tuple(k_raw.shape), device)
    rows = k_raw.numel() // dk if dk else 0
    rc = L.ckda_prep(_ptr(q_raw), _ptr(k_raw), _ptr(a_raw), _ptr(b_raw), _ptr(q), _ptr(k),
                     _ptr(alpha), _ptr(beta), int(rows), int(dk), _io_dtype(k_raw),
                     int(bool(normalize_q)), float(norm_eps), _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_prep")
    return q, k, alpha, beta


def prep_bwd(k_raw, a_raw, b_raw, d_k, d_alpha, d_beta, q_raw=None, d_q=None, normalize_q=True,
             norm_eps=1e-6, out=None, stream=None):
    """Backward of ``prep`` (ckda_prep_bwd): the gradients with respect to the
    raw inputs from those with respect to (q, k, alpha, beta).  The gate's
    sign carries no gradient and |tanh(a/2)| takes the subgradient 0 at a = 0.

    Returns (d_q_raw or None, d_k_raw, d_a_raw, d_b_raw) in the input dtype;
    `out` may give the four output tensors (d_q_raw may be None)."""
    if stream is not None:
        return _on_stream(prep_bwd, locals())
    L = lib()
    device = k_raw.device
    dt = k_raw.dtype
    shp = tuple(k_raw.shape)
    dk = shp[-1]
    for name, t, want in (("a_raw", a_raw, shp), ("b_raw", b_raw, shp[:-1]), ("d_k", d_k, shp),
                          ("d_alpha", d_alpha, shp), ("d_beta", d_beta, shp[:-1]),
                          ("k_raw", k_raw, shp)):
        _check(t, name, dt, want, device)
    if (q_raw is None) != (d_q is None):
        raise ValueError("prep_bwd: q_raw and d_q must both be given or both be None")
    if q_raw is not None:
        _check(q_raw, "q_raw", dt, shp, device)
        _check(d_q, "d_q", dt, shp, device)
    if out is None:
        dq_raw = None if q_raw is None else torch.empty_like(q_raw)
        dk_raw, da_raw, db_raw = (torch.empty_like(k_raw), torch.empty_like(a_raw),
                                  torch.empty_like(b_raw))
    else:
        dq_raw, dk_raw, da_raw, db_raw = out
        for name, t, want in (("d_k_raw", dk_raw, shp), ("d_a_raw", da_raw, shp),
                              ("d_b_raw", db_raw, shp[:-1])):
            _check(t, name, dt, want, device)
        if (dq_raw is None) != (q_raw is None):
            raise ValueError("prep_bwd: d_q_raw and q_raw must both be given or both be None")
        if dq_raw is not None:
            _check(dq_raw, "d_q_raw", dt, shp, device)
    rows = k_raw.numel() // dk if dk else 0
    rc = L.ckda_prep_bwd(_ptr(q_raw), _ptr(k_raw), _ptr(a_raw), _ptr(b_raw), _ptr(d_q),
                         _ptr(d_k), _ptr(d_alpha), _ptr(d_beta), _ptr(dq_raw), _ptr(dk_raw),
                         _ptr(da_raw), _ptr(db_raw), int(rows), int(dk), _io_dtype(k_raw),
                         int(bool(normalize_q)), float(norm_eps), _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_prep_bwd")
    return dq_raw, dk_raw, da_raw, db_raw


def bwd_workspace_bytes(B, H, T, dk, dv, num_seqs=0) -> int:
    return int(lib().ckda_bwd_workspace_bytes(num_seqs, B, H, T, dk, dv))


def bwd(q, k, v, alpha, beta, do, h0=None, dhT=None, cu_seqlens=None, scale=1.0,
        store_dh0=True, workspace=None, stream=None):
    """Backward of fwd (ckda_bwd): gradients of sum <o, do> + <hT, dhT>.

    Returns (dq, dk, dv, dalpha, dbeta, dh0 or None); dh0 is fp32."""
    if stream is not None:
        return _on_stream(bwd, locals())
    L = lib()
    device = q.device
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _io_dtype(q)
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)),
                         ("alpha", alpha, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("do", do, (B, H, T, dv)), ("beta", beta, (B, H, T))):
        _check(t, name, dt, shp, device)
    N = B
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), device)
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _check(t, name, torch.float32, (N, H, dk, dv), device)
    need = bwd_workspace_bytes(B, H, T, dk, dv, N if cu_seqlens is not None else 0)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    dq, dkk, dal = torch.empty_like(q), torch.empty_like(k), torch.empty_like(alpha)
    dvv, dbe = torch.empty_like(v), torch.empty_like(beta)
    dh0 = torch.empty((N, H, dk, dv), dtype=torch.float32, device=device) if store_dh0 else None
    rc = L.ckda_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(do),
                    _ptr(dhT), _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dal), _ptr(dbe), _ptr(dh0),
                    _ptr(cu_seqlens), int(N if cu_seqlens is not None else 0), B, H, T, dk, dv,
                    _io_dtype(q), float(scale), _ptr(workspace), _given(workspace, device),
                    _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_bwd")
    return dq, dkk, dvv, dal, dbe, dh0


def decode_step_raw(q_raw, k_raw, v, a_raw, b_raw, state, scale=1.0, normalize_q=True,
                    norm_eps=1e-6, o=None, stream=None):
    """One decode step on raw inputs with the input preparation fused in
    (ckda_decode_step_raw): unit-norm k (and q), alpha and beta from the gate
    logits a and b.  state [B, H, 128, 128] fp32 is updated in place; returns o."""
    if stream is not None:
        return _on_stream(decode_step_raw, locals())
    L = lib()
    device = q_raw.device
    B, H, dk = q_raw.shape
    dv = v.shape[-1]
    dt = q_raw.dtype
    for name, t, shp in (("q_raw", q_raw, (B, H, dk)), ("k_raw", k_raw, (B, H, dk)),
                         ("a_raw", a_raw, (B, H, dk)), ("v", v, (B, H, dv)),
                         ("b_raw", b_raw, (B, H))):
        _check(t, name, dt, shp, device)
    _check(state, "state", torch.float32, (B, H, dk, dv), device)
    if o is None:
        o = torch.empty((B, H, dv), dtype=dt, device=device)
    else:
        _check(o, "o", dt, (B, H, dv), device)
    rc = L.ckda_decode_step_raw(_ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(a_raw), _ptr(b_raw),
                                _ptr(state), _ptr(o), B, H, dk, dv, _io_dtype(q_raw),
                                float(scale), int(bool(normalize_q)), float(norm_eps),
                                _stream_handle(None, device))
    if rc != 0:
        raise CkdaError(rc, "ckda_decode_step_raw")
    return o


# What the calls below share.  A single token or a few rows take the GPU a few
# microseconds, so the host's part is kept short: plain addresses, and the
# device switched only when it is another.
def _addr(t):
    return None if t is None else t.data_ptr()


def _call(fn, where, device, *args):
    """fn(*args, current stream) on the tensors' device; raises CkdaError."""
    if device.type != "cuda":
        raise ValueError(f"tensors on {device}, expected CUDA")
    handle = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch._C._cuda_getDevice():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc != 0:
        raise CkdaError(rc, where)


@functools.lru_cache(maxsize=4096)
def _bytes(name, *args):
    return int(getattr(lib(), name)(*args))


# ------------------------------------ linear attention with a decay per head
def _check_linear(q, k, v, g, cu_seqlens, states, more=()):
    """Checks the arguments that linear_fwd and linear_bwd share; returns
    (B, H, Hk, T, dk, dv, N, g per head, io dtype)."""
    device, dt = q.device, q.dtype
    io = _io_dtype(q)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q [B, Hk, T, dk] and v [B, H, T, dv] have four axes")
    B, Hk, T, dk = q.shape
    H, dv = v.shape[1], v.shape[3]
    if Hk < 1 or H % Hk:
        raise ValueError(f"{H} heads cannot share {Hk} key heads evenly")
    _check(q, "q", dt, (B, Hk, T, dk), device)
    _check(k, "k", dt, (B, Hk, T, dk), device)
    _check(v, "v", dt, (B, H, T, dv), device)
    for name, t in more:
        _check(t, name, dt, (B, H, T, dv), device)
    per_head = g.dim() == 1
    _check(g, "g", torch.float32, (H,) if per_head else (B, H, T), device)
    N = B
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or B != 1:
            raise ValueError("packed input has B = 1 and cu_seqlens [num_seqs + 1]")
        N = cu_seqlens.numel() - 1
        _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), device)
    for name, t in states:
        if t is not None:
            _check(t, name, torch.float32, (N, H, dk, dv), device)
    return B, H, Hk, T, dk, dv, N, per_head, io


# A call's last_workspace is for fwd_status.  What the call made for itself is given back before
# the next is made where it is more than _SMALL, and at the call's end, all but the status word,
# where it is more than _LARGE: that copy takes 4 us, a call on so much memory over a
# millisecond (on 268 MB, the backward of 8 x 16 x 2048, it would be 272 us and 276).
_SMALL, _LARGE = 1 << 20, 1 << 30


def linear_fwd_workspace_bytes(B, H, T, dk, dv, dtype=torch.bfloat16, num_seqs=0) -> int:
    io = _BF16 if dtype == torch.bfloat16 else _F32
    return _bytes("ckda_linear_fwd_workspace_bytes", num_seqs, B, H, T, dk, dv, io)


def linear_bwd_workspace_bytes(B, H, Hk, T, dk, dv, dtype=torch.bfloat16, num_seqs=0) -> int:
    io = _BF16 if dtype == torch.bfloat16 else _F32
    return _bytes("ckda_linear_bwd_workspace_bytes", num_seqs, B, H, Hk, T, dk, dv, io)


def linear_fwd(q, k, v, g, h0=None, cu_seqlens=None, scale=1.0, store_final_state=True, o=None,
               hT=None, workspace=None, stream=None):
    """Linear attention with a scalar decay per head (ckda_linear_fwd):
    H_t = exp(g_t) H_{t-1} + k_t v_t^T, o_t = H_t^T (scale q_t).

    q, k [B, Hk, T, dk] with Hk dividing H (heads share keys in order),
    v [B, H, T, dv], g fp32 [B, H, T] or [H] (one decay for all of a head's
    tokens); h0, hT fp32 [N, H, dk, dv].  Returns (o, hT or None)."""
    if stream is not None:
        return _on_stream(linear_fwd, locals())
    L = lib()
    device = q.device
    B, H, Hk, T, dk, dv, N, per_head, io = _check_linear(q, k, v, g, cu_seqlens,
                                                         (("h0", h0), ("hT", hT)))
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=q.dtype, device=device)
    else:
        _check(o, "o", q.dtype, (B, H, T, dv), device)
    if store_final_state and hT is None:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=device)
    nseq = N if cu_seqlens is not None else 0
    pq, pk, pv, po = q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr()
    own = workspace is None
    if own:
        size = _bytes("ckda_linear_fwd_workspace_bytes" if (pq | pk | pv | po) & 15 else
                      "ckda_linear_fwd_aligned_workspace_bytes", nseq, B, H, T, dk, dv, io)
        if size > _SMALL:
            linear_fwd.last_workspace = None
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        size = _given(workspace, device)
    _call(L.ckda_linear_fwd, "ckda_linear_fwd", device, pq, pk, pv, g.data_ptr(), int(per_head),
          _addr(h0), po, _addr(hT), _addr(cu_seqlens), nseq, B, H, Hk, T, dk, dv, io, float(scale),
          workspace.data_ptr(), size)
    linear_fwd.last_workspace = workspace[:256].clone() if own and size > _LARGE else workspace
    return o, hT


def linear_bwd(q, k, v, g, do, h0=None, dhT=None, cu_seqlens=None, scale=1.0, store_dh0=True,
               workspace=None, stream=None):
    """Backward of linear_fwd (ckda_linear_bwd): gradients of
    sum <o, do> + <hT, dhT>.  Returns (dq, dk, dv, dg, dh0 or None); dg (of g's
    shape) and dh0 are fp32."""
    if stream is not None:
        return _on_stream(linear_bwd, locals())
    L = lib()
    device = q.device
    B, H, Hk, T, dk, dv, N, per_head, io = _check_linear(q, k, v, g, cu_seqlens,
                                                         (("h0", h0), ("dhT", dhT)), (("do", do),))
    nseq = N if cu_seqlens is not None else 0
    pq, pk, pv, pdo = q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr()
    own = workspace is None
    if own:
        size = _bytes("ckda_linear_bwd_workspace_bytes" if (pq | pk | pv | pdo) & 15 else
                      "ckda_linear_bwd_aligned_workspace_bytes", nseq, B, H, Hk, T, dk, dv, io)
        if size > _SMALL:
            linear_bwd.last_workspace = None
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        size = _given(workspace, device)
    dq, dkk, dvv, dg = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                        torch.empty_like(g))
    dh0 = torch.empty((N, H, dk, dv), dtype=torch.float32, device=device) if store_dh0 else None
    _call(L.ckda_linear_bwd, "ckda_linear_bwd", device, pq, pk, pv, g.data_ptr(), int(per_head),
          _addr(h0), pdo, _addr(dhT), dq.data_ptr(), dkk.data_ptr(), dvv.data_ptr(), dg.data_ptr(),
          _addr(dh0), _addr(cu_seqlens), nseq, B, H, Hk, T, dk, dv, io, float(scale),
          workspace.data_ptr(), size)
    linear_bwd.last_workspace = workspace[:256].clone() if own and size > _LARGE else workspace
    return dq, dkk, dvv, dg, dh0


def linear_decode_step(q, k, v, g, state, scale=1.0, o=None, stream=None):
    """One token of linear attention (ckda_linear_decode_step) on a resident
    state [B, H, dk, dv] fp32, updated in place.  q, k [B, Hk, dk],
    v [B, H, dv], g fp32 [B, H] or [H].  Returns o [B, H, dv]."""
    if stream is not None:
        return _on_stream(linear_decode_step, locals())
    L = lib()
    device, dt = q.device, q.dtype
    io = _io_dtype(q)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q [B, Hk, dk] and v [B, H, dv] have three axes")
    B, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    if Hk < 1 or H % Hk:
        raise ValueError(f"{H} heads cannot share {Hk} key heads evenly")
    _check(q, "q", dt, (B, Hk, dk), device)
    _check(k, "k", dt, (B, Hk, dk), device)
    _check(v, "v", dt, (B, H, dv), device)
    per_head = g.dim() == 1
    _check(g, "g", torch.float32, (H,) if per_head else (B, H), device)
    _check(state, "state", torch.float32, (B, H, dk, dv), device)
    if o is None:
        o = torch.empty((B, H, dv), dtype=dt, device=device)
    else:
        _check(o, "o", dt, (B, H, dv), device)
    _call(L.ckda_linear_decode_step, "ckda_linear_decode_step", device, _addr(q),
          _addr(k), _addr(v), _addr(g), int(per_head), _addr(state), _addr(o), B, H, Hk, dk, dv,
          io, float(scale))
    return o


# ----------------------------------------------------------------- layer norm
def _check_weight(weight, bias, width, device):
    """The weights' dtype code (fp32 when there are none)."""
    wt = weight if weight is not None else bias
    if wt is None:
        return _F32
    code = _io_dtype(wt)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check(t, name, wt.dtype, (width,), device)
    return code


def layernorm_fwd(x, weight=None, bias=None, eps=1e-5, y=None, mean=None, rstd=None, stream=None):
    """Layer norm over the last axis (ckda_layernorm_fwd).  Returns (y, mean,
    rstd); mean and rstd are fp32 of x's leading shape.  weight and bias are
    bf16 or fp32 [width], whatever x's type.  y may be x (in place)."""
    if stream is not None:
        return _on_stream(layernorm_fwd, locals())
    L = lib()
    device = x.device
    io = _io_dtype(x)
    if x.dim() < 1:
        raise ValueError("x has no last axis")
    lead, width = x.shape[:-1], x.shape[-1]
    if not x.is_contiguous():
        raise ValueError("x: must be contiguous")
    wcode = _check_weight(weight, bias, width, device)
    if y is None:
        y = torch.empty_like(x)
    else:
        _check(y, "y", x.dtype, x.shape, device)
    if mean is None:
        mean = torch.empty(lead, dtype=torch.float32, device=device)
    else:
        _check(mean, "mean", torch.float32, lead, device)
    if rstd is None:
        rstd = torch.empty(lead, dtype=torch.float32, device=device)
    else:
        _check(rstd, "rstd", torch.float32, lead, device)
    _call(L.ckda_layernorm_fwd, "ckda_layernorm_fwd", device, _addr(x), _addr(weight),
          _addr(bias), _addr(y), _addr(mean), _addr(rstd), mean.numel(), width, io, wcode,
          float(eps))
    return y, mean, rstd


def layernorm_bwd(dy, x, mean, rstd, weight=None, weight_grad=True, dx=None, workspace=None,
                  stream=None):
    """Backward of layernorm_fwd (ckda_layernorm_bwd).  Returns (dx, dweight,
    dbias); the last two have weight's type (fp32 without one) and are None
    when weight_grad is false.  dx may be dy or x (in place)."""
    if stream is not None:
        return _on_stream(layernorm_bwd, locals())
    L = lib()
    device = x.device
    io = _io_dtype(x)
    if x.dim() < 1:
        raise ValueError("x has no last axis")
    lead, width = x.shape[:-1], x.shape[-1]
    if not x.is_contiguous():
        raise ValueError("x: must be contiguous")
    _check(dy, "dy", x.dtype, x.shape, device)
    _check(mean, "mean", torch.float32, lead, device)
    _check(rstd, "rstd", torch.float32, lead, device)
    wcode = _check_weight(weight, None, width, device)
    if dx is None:
        dx = torch.empty_like(x)
    else:
        _check(dx, "dx", x.dtype, x.shape, device)
    rows = mean.numel()
    dw = db = None
    if weight_grad:
        wdt = torch.float32 if weight is None else weight.dtype
        dw = torch.empty(width, dtype=wdt, device=device)
        db = torch.empty(width, dtype=wdt, device=device)
        if workspace is None:
            workspace = torch.empty(_bytes("ckda_layernorm_bwd_workspace_bytes", rows, width),
                                    dtype=torch.uint8, device=device)
    _call(L.ckda_layernorm_bwd, "ckda_layernorm_bwd", device, _addr(dy), _addr(x),
          _addr(mean), _addr(rstd), _addr(weight), _addr(dx), _addr(dw), _addr(db), rows, width,
          io, wcode, _addr(workspace),
          0 if workspace is None else _given(workspace, device))
    return dx, dw, db


# ----------------------------------------- short convolution and selective scan
def _apart(t, name, dtype, shape, device, tail=1):
    """Checks rows of the last `tail` axes: each row in one run, rows evenly apart (a part
    of a wider projection).  Returns the elements from one row to the next."""
    if t.is_contiguous() and t.dtype == dtype and t.shape == shape and t.device == device:
        return shape[-1] if tail == 1 else shape[-1] * shape[-2]
    if t.dtype != dtype or t.shape != shape or t.device != device:
        _check(t, name, dtype, shape, device)
    width = 1
    strides = t.stride()
    for i in range(len(shape) - 1, len(shape) - 1 - tail, -1):
        if shape[i] > 1 and strides[i] != width:
            raise ValueError(f"{name}: each row must be contiguous")
        width *= shape[i]
    apart, rows = None, 1
    for i in range(len(shape) - 1 - tail, -1, -1):
        if shape[i] > 1:
            if apart is None:
                apart = strides[i]
            if strides[i] != apart * rows or apart < width:
                raise ValueError(f"{name}: rows must be evenly apart and not overlap")
            rows *= shape[i]
    return width if apart is None else apart


def _like(x, shape=None, dtype=None):
    """New memory of x's (or another) shape and type.  (empty_like takes less than half of
    empty's time, which is a tenth of a single token's call.)"""
    if shape is None:
        if x.is_contiguous():
            return torch.empty_like(x) if dtype is None else torch.empty_like(x, dtype=dtype)
        shape = x.shape
    return x.new_empty(shape) if dtype is None else x.new_empty(shape, dtype=dtype)


def _sequences(B, cu_seqlens, device):
    """Sequences of the states, and the count that the library takes."""
    if cu_seqlens is None:
        return B, 0
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or B != 1:
        raise ValueError("packed input has B = 1 and cu_seqlens [num_seqs + 1]")
    n = cu_seqlens.numel() - 1
    _check(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), device)
    return n, n


def _check_conv(x, weight, bias, axes):
    """(io code, weight code, rows' distance, taps) of what the convolution's calls share."""
    if x.dim() != axes:
        raise ValueError(f"x [{'B, T, D' if axes == 3 else 'B, D'}] has {axes} axes")
    io = _io_dtype(x)
    if weight.dim() != 2:
        raise ValueError("weight [D, W] has two axes")
    code = _io_dtype(weight)
    D, W = x.shape[-1], weight.shape[1]
    device = x.device
    _check(weight, "weight", weight.dtype, (D, W), device)
    if bias is not None:
        _check(bias, "bias", weight.dtype, (D,), device)
    return io, code, D if x.is_contiguous() else _apart(x, "x", x.dtype, x.shape, device), W


def conv_fwd(x, weight, bias=None, h0=None, cu_seqlens=None, silu=True, store_final_state=True,
             y=None, hT=None, stream=None):
    """Short causal convolution of each channel (ckda_conv_fwd): p_t = bias +
    sum_j weight_j x_{t-W+1+j}, y = silu(p) or, with silu=False, p.

    x [B, T, D] (it may be a part of a wider projection's last axis), weight [D, W] with
    W = 2, 3 or 4 and bias [D] in bf16 or fp32, h0, hT [N, W - 1, D] in x's type: the inputs
    before the first token and the last ones.  Packed sequences may end before T: rows behind
    the last one are not read, and zero in y (a y that is given keeps its own there).
    Returns (y, hT or None)."""
    if stream is not None:
        return _on_stream(conv_fwd, locals())
    L = lib()
    device, dt = x.device, x.dtype
    io, code, ldx, W = _check_conv(x, weight, bias, 3)
    B, T, D = x.shape
    N, nseq = _sequences(B, cu_seqlens, device)
    if h0 is not None:
        _check(h0, "h0", dt, (N, W - 1, D), device)
    call = L.ckda_conv_fwd
    if y is None:
        y = _like(x)
        if nseq:
            call = L.ckda_conv_fwd_filled
    else:
        _check(y, "y", dt, (B, T, D), device)
    if hT is not None:
        _check(hT, "hT", dt, (N, W - 1, D), device)
    elif store_final_state:
        hT = _like(x, (N, W - 1, D))
    _call(call, "ckda_conv_fwd", device, x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(h0),
          y.data_ptr(), _addr(hT), _addr(cu_seqlens), nseq, B, T, D, W, ldx, io, code, int(silu))
    return y, hT


def conv_bwd(dy, x, weight, bias=None, h0=None, dhT=None, cu_seqlens=None, silu=True,
             store_dh0=True, workspace=None, stream=None):
    """Backward of conv_fwd (ckda_conv_bwd): gradients of sum <y, dy> + <hT, dhT>.  Returns
    (dx, dweight, dbias or None, dh0 or None); the weights' have the weights' type; dx is zero
    in rows behind the last packed sequence."""
    if stream is not None:
        return _on_stream(conv_bwd, locals())
    L = lib()
    device, dt = x.device, x.dtype
    io, code, ldx, W = _check_conv(x, weight, bias, 3)
    B, T, D = x.shape
    N, nseq = _sequences(B, cu_seqlens, device)
    _check(dy, "dy", dt, (B, T, D), device)
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _check(t, name, dt, (N, W - 1, D), device)
    if workspace is None:
        size = _bytes("ckda_conv_bwd_workspace_bytes", B, T, D, W)
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        size = _given(workspace, device)
    dx = _like(x)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dh0 = _like(x, (N, W - 1, D)) if store_dh0 else None
    _call(L.ckda_conv_bwd, "ckda_conv_bwd", device, dy.data_ptr(), x.data_ptr(), weight.data_ptr(),
          _addr(bias), _addr(h0), _addr(dhT), dx.data_ptr(), dw.data_ptr(), _addr(db), _addr(dh0),
          _addr(cu_seqlens), nseq, B, T, D, W, ldx, io, code, int(silu), workspace.data_ptr(), size)
    return dx, dw, db, dh0


def conv_decode_step(x, weight, state, bias=None, silu=True, y=None, stream=None):
    """One token of the convolution (ckda_conv_decode_step): x [B, D]; state [B, W - 1, D] in
    x's type is moved on by the token in place.  Returns y [B, D]."""
    if stream is not None:
        return _on_stream(conv_decode_step, locals())
    L = lib()
    device, dt = x.device, x.dtype
    io, code, ldx, W = _check_conv(x, weight, bias, 2)
    B, D = x.shape
    _check(state, "state", dt, (B, W - 1, D), device)
    if y is None:
        y = _like(x)
    else:
        _check(y, "y", dt, (B, D), device)
    _call(L.ckda_conv_decode_step, "ckda_conv_decode_step", device, x.data_ptr(), weight.data_ptr(),
          _addr(bias), state.data_ptr(), y.data_ptr(), B, D, W, ldx, io, code, int(silu))
    return y


def _check_scan(x, dt, A, B, C, D, z, dt_bias, axes):
    """Checks what the scan's calls share; returns (io, N, G, distances of x, dt, B, C, z)."""
    if x.dim() != axes:
        raise ValueError(f"x [{'B, T, D' if axes == 3 else 'B, D'}] has {axes} axes")
    io, device, t, shape = _io_dtype(x), x.device, x.dtype, x.shape
    width = shape[-1]
    if A.dim() != 2:
        raise ValueError("A [D, N] has two axes")
    N = A.shape[1]
    _check(A, "A", torch.float32, (width, N), device)
    rank = B.dim()
    if rank not in (axes, axes + 1) or rank != C.dim():
        raise ValueError("B and C are both [..., N] or both [..., G, N]")
    G = B.shape[-2] if rank > axes else 1
    if G < 1 or width % G:
        raise ValueError(f"{width} channels cannot share {G} groups evenly")
    tail = 1 + rank - axes
    groups = (*shape[:-1], G, N) if tail == 2 else (*shape[:-1], N)
    if D is not None:
        _check(D, "D", torch.float32, (width,), device)
    if dt_bias is not None:
        _check(dt_bias, "dt_bias", torch.float32, (width,), device)
    return io, N, G, (width if x.is_contiguous() else _apart(x, "x", t, shape, device),
                      _apart(dt, "dt", t, shape, device), _apart(B, "B", t, groups, device, tail),
                      _apart(C, "C", t, groups, device, tail),
                      0 if z is None else _apart(z, "z", t, shape, device))


def scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None,
             softplus=True, store_final_state=True, y=None, hT=None, workspace=None, stream=None):
    """Selective state space scan (ckda_scan_fwd): delta = softplus(dt + dt_bias),
    h_t = exp(delta A) h_{t-1} + delta x B_t, y_t = (<C_t, h_t> + D x_t) silu(z_t).

    x, dt, z [B, T, D]; B, C [B, T, N], or [B, T, G, N] with G dividing D; each may be a part
    of a wider projection's last axis.  A fp32 [D, N], N <= 64; D, dt_bias fp32 [D]; h0, hT
    fp32 [sequences, D, N].  Packed sequences may end before T: rows behind the last one are
    not read, and zero in y (a y that is given keeps its own there).  Returns (y, hT or None)."""
    if stream is not None:
        return _on_stream(scan_fwd, locals())
    L = lib()
    device = x.device
    io, N, G, apart = _check_scan(x, dt, A, B, C, D, z, dt_bias, 3)
    rows, T, width = x.shape
    count, nseq = _sequences(rows, cu_seqlens, device)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (count, width, N), device)
    call = L.ckda_scan_fwd
    if y is None:
        y = _like(x)
        if nseq:
            call = L.ckda_scan_fwd_filled
    else:
        _check(y, "y", x.dtype, (rows, T, width), device)
    if hT is not None:
        _check(hT, "hT", torch.float32, (count, width, N), device)
    elif store_final_state:
        hT = _like(A, (count, width, N)) if h0 is None else torch.empty_like(h0)
    if workspace is None:
        size = _bytes("ckda_scan_fwd_workspace_bytes", rows, T, width, N, G)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        size = _given(workspace, device)
    _call(call, "ckda_scan_fwd", device, x.data_ptr(), dt.data_ptr(), A.data_ptr(),
          B.data_ptr(), C.data_ptr(), _addr(D), _addr(z), _addr(dt_bias), _addr(h0), y.data_ptr(),
          _addr(hT), _addr(cu_seqlens), nseq, rows, T, width, N, G, *apart, io, int(softplus),
          _addr(workspace), size)
    return y, hT


def scan_bwd(dy, x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, dhT=None, cu_seqlens=None,
             softplus=True, store_dh0=True, workspace=None, stream=None):
    """Backward of scan_fwd (ckda_scan_bwd): gradients of sum <y, dy> + <hT, dhT>.  Returns
    (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0); those of what was not given are None, those
    by token zero in rows behind the last packed sequence.  Its workspace has about a byte for
    every token, channel and state."""
    if stream is not None:
        return _on_stream(scan_bwd, locals())
    L = lib()
    device, f32 = x.device, torch.float32
    io, N, G, apart = _check_scan(x, dt, A, B, C, D, z, dt_bias, 3)
    rows, T, width = x.shape
    count, nseq = _sequences(rows, cu_seqlens, device)
    _check(dy, "dy", x.dtype, x.shape, device)
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _check(t, name, f32, (count, width, N), device)
    if workspace is None:
        size = _bytes("ckda_scan_bwd_workspace_bytes", rows, T, width, N, G)
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        size = _given(workspace, device)

    dx, ddt, dA, dB, dC, dD, dz, ddt_bias = (None if t is None else _like(t)
                                             for t in (x, dt, A, B, C, D, z, dt_bias))
    dh0 = _like(A, (count, width, N)) if store_dh0 else None
    _call(L.ckda_scan_bwd, "ckda_scan_bwd", device, dy.data_ptr(), x.data_ptr(), dt.data_ptr(),
          A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D), _addr(z), _addr(dt_bias), _addr(h0),
          _addr(dhT), dx.data_ptr(), ddt.data_ptr(), dA.data_ptr(), dB.data_ptr(), dC.data_ptr(),
          _addr(dD), _addr(dz), _addr(ddt_bias), _addr(dh0), _addr(cu_seqlens), nseq, rows, T,
          width, N, G, *apart, io, int(softplus), workspace.data_ptr(), size)
    return dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0


def scan_decode_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus=True, y=None,
                     stream=None):
    """One token of the scan (ckda_scan_decode_step) on a resident state [B, D, N] fp32,
    updated in place.  x, dt, z [B, D]; B, C [B, N] or [B, G, N].  Returns y [B, D]."""
    if stream is not None:
        return _on_stream(scan_decode_step, locals())
    L = lib()
    device = x.device
    io, N, G, apart = _check_scan(x, dt, A, B, C, D, z, dt_bias, 2)
    rows, width = x.shape
    _check(state, "state", torch.float32, (rows, width, N), device)
    if y is None:
        y = _like(x)
    else:
        _check(y, "y", x.dtype, (rows, width), device)
    _call(L.ckda_scan_decode_step, "ckda_scan_decode_step", device, x.data_ptr(), dt.data_ptr(),
          A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D), _addr(z), _addr(dt_bias),
          state.data_ptr(), y.data_ptr(), rows, width, N, G, *apart, io, int(softplus))
    return y


# ------------------------------------------------------------------- RMS norm
def _check_rms(x, weight, residual):
    """(io code, weight code, leading shape, width, sum's tensor or None)."""
    io = _io_dtype(x)
    if x.dim() < 1:
        raise ValueError("x has no last axis")
    if not x.is_contiguous():
        raise ValueError("x: must be contiguous")
    code = _check_weight(weight, None, x.shape[-1], x.device)
    if residual is not None:
        _check(residual, "residual", x.dtype, x.shape, x.device)
    return io, code, x.shape[:-1], x.shape[-1]


def rmsnorm_fwd(x, weight=None, residual=None, eps=1e-5, y=None, h=None, rstd=None, stream=None):
    """Root-mean-square norm over the last axis of h = x + residual (ckda_rmsnorm_fwd).
    Returns (y, h, rstd): h is x itself without a residual; rstd is fp32 of x's leading
    shape.  residual has x's type; weight is bf16 or fp32 [width].  h and y may each be x or
    residual, not the same (y=x without a residual leaves no h for rmsnorm_bwd)."""
    if stream is not None:
        return _on_stream(rmsnorm_fwd, locals())
    L = lib()
    device = x.device
    io, code, lead, width = _check_rms(x, weight, residual)
    if y is None:
        y = torch.empty_like(x)
    else:
        _check(y, "y", x.dtype, x.shape, device)
    if residual is None:
        if h is not None:
            raise ValueError("h: there is no sum to store without a residual")
    elif h is None:
        h = torch.empty_like(x)
    else:
        _check(h, "h", x.dtype, x.shape, device)
    if rstd is None:
        rstd = _like(x, lead, torch.float32)
    else:
        _check(rstd, "rstd", torch.float32, lead, device)
    _call(L.ckda_rmsnorm_fwd, "ckda_rmsnorm_fwd", device, x.data_ptr(), _addr(residual),
          _addr(weight), _addr(h), y.data_ptr(), rstd.data_ptr(), rstd.numel(), width, io, code,
          float(eps))
    return y, x if h is None else h, rstd


def rmsnorm_fwd8(x, weight=None, residual=None, eps=1e-5, group=0, stream=None):
    """rmsnorm_fwd with y in 8 bits (ckda_rmsnorm_fwd8).  Returns (y8, scale, h, rstd): y8 is
    float8_e4m3fn and y = y8 scale; scale is fp32 of x's leading shape (group = 0: one for a
    row), or with a last axis of width / group (group = 32, 64 or 128 columns each).  It is
    for a product in 8 bits of the user's; the library has none."""
    if stream is not None:
        return _on_stream(rmsnorm_fwd8, locals())
    L = lib()
    device = x.device
    io, code, lead, width = _check_rms(x, weight, residual)
    if group and (group not in (32, 64, 128) or width % group):
        raise ValueError(f"group: {group}, expected 0, 32, 64 or 128 that divides {width}")
    y8 = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    h = None if residual is None else torch.empty_like(x)
    rstd = _like(x, lead, torch.float32)
    scale = _like(x, (*lead, width // group), torch.float32) if group else torch.empty_like(rstd)
    _call(L.ckda_rmsnorm_fwd8, "ckda_rmsnorm_fwd8", device, x.data_ptr(), _addr(residual),
          _addr(weight), _addr(h), y8.data_ptr(), scale.data_ptr(), rstd.data_ptr(), rstd.numel(),
          width, int(group), io, code, float(eps))
    return y8, scale, x if h is None else h, rstd


def rmsnorm_bwd(dy, h, rstd, weight=None, dh=None, weight_grad=True, dx=None, workspace=None,
                stream=None):
    """Backward of rmsnorm_fwd and rmsnorm_fwd8 (ckda_rmsnorm_bwd), from the h and rstd that
    they returned; dh is the gradient that arrives at h itself.  Returns (dx, dweight): dx is
    the gradient of x and of residual alike; dweight has weight's type (fp32 without one) and
    is None when weight_grad is false.  dx may be dy, h or dh."""
    if stream is not None:
        return _on_stream(rmsnorm_bwd, locals())
    L = lib()
    device = h.device
    io, code, lead, width = _check_rms(h, weight, None)
    _check(dy, "dy", h.dtype, h.shape, device)
    _check(rstd, "rstd", torch.float32, lead, device)
    if dh is not None:
        _check(dh, "dh", h.dtype, h.shape, device)
    if dx is None:
        dx = torch.empty_like(h)
    else:
        _check(dx, "dx", h.dtype, h.shape, device)
    rows, dw = rstd.numel(), None
    if weight_grad:
        dw = _like(rstd, (width,)) if weight is None else torch.empty_like(weight)
        if workspace is None:
            workspace = torch.empty(_bytes("ckda_rmsnorm_bwd_workspace_bytes", rows, width),
                                    dtype=torch.uint8, device=device)
    _call(L.ckda_rmsnorm_bwd, "ckda_rmsnorm_bwd", device, dy.data_ptr(), h.data_ptr(),
          rstd.data_ptr(), _addr(weight), _addr(dh), dx.data_ptr(), _addr(dw), rows, width, io, code,
          _addr(workspace), 0 if workspace is None else _given(workspace, device))
    return dx, dw


# ------------------------------------------------------------------- autograd
# Training use: the forward (fwd) with its backward (bwd), and the input
# preparation (prep) with its backward (prep_bwd), as torch.autograd
# functions.  They only route tensors between the calls above.
#
# None has a second derivative.  Where one would be needed (create_graph=True), the gradients
# are tied to whatever they depend on, with an error in place of a derivative; without the tie
# they would count as constants.
class _NoDerivative(torch.autograd.Function):
    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of this library's calls have no second derivative")


def _once(backward):
    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        with torch.no_grad():
            outs = list(backward(ctx, *grads))
        if torch.is_grad_enabled():
            have = [i for i, t in enumerate(outs) if t is not None]
            behind = [t for t in (*grads, *ctx.saved_tensors) if t is not None]
            tied = _NoDerivative.apply(len(have), *(outs[i] for i in have), *behind)
            for i, t in zip(have, tied):
                outs[i] = t
        return tuple(outs)
    return wrapped


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, alpha, beta, h0, cu_seqlens, scale):
        o, hT = fwd(q, k, v, alpha, beta, h0, cu_seqlens, scale=scale)
        ctx.save_for_backward(q, k, v, alpha, beta, h0, cu_seqlens)
        ctx.scale = scale
        return o, hT

    @staticmethod
    @_once
    def backward(ctx, do, dhT):
        q, k, v, alpha, beta, h0, cu = ctx.saved_tensors
        do = torch.zeros_like(v) if do is None else do.contiguous()
        dhT = None if dhT is None else dhT.contiguous()
        dq, dk, dv, da, db, dh0 = bwd(q, k, v, alpha, beta, do, h0=h0, dhT=dhT, cu_seqlens=cu,
                                      scale=ctx.scale, store_dh0=h0 is not None)
        return dq, dk, dv, da, db, dh0, None, None


def recurrence(q, k, v, alpha, beta, h0=None, cu_seqlens=None, scale=1.0):
    """(o, hT) = fwd(...), differentiable in q, k, v, alpha, beta and h0
    (the gradients come from bwd).  hT is fp32 [N, H, dk, dv]."""
    return _Recurrence.apply(q, k, v, alpha, beta, h0, cu_seqlens, float(scale))


class _Prepare(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q_raw, k_raw, a_raw, b_raw, normalize_q, norm_eps):
        q, k, alpha, beta = prep(k_raw, a_raw, b_raw, q_raw=q_raw, normalize_q=normalize_q,
                                 norm_eps=norm_eps)
        ctx.save_for_backward(q_raw, k_raw, a_raw, b_raw)
        ctx.normalize_q, ctx.norm_eps = normalize_q, norm_eps
        return q, k, alpha, beta

    @staticmethod
    @_once
    def backward(ctx, dq, dk, dalpha, dbeta):
        q_raw, k_raw, a_raw, b_raw = ctx.saved_tensors
        z = lambda g, like: torch.zeros_like(like) if g is None else g.contiguous()
        dq_raw, dk_raw, da_raw, db_raw = prep_bwd(
            k_raw, a_raw, b_raw, z(dk, k_raw), z(dalpha, a_raw), z(dbeta, b_raw), q_raw=q_raw,
            d_q=z(dq, q_raw), normalize_q=ctx.normalize_q, norm_eps=ctx.norm_eps)
        return dq_raw, dk_raw, da_raw, db_raw, None, None


def prepare(q_raw, k_raw, a_raw, b_raw, normalize_q=True, norm_eps=1e-6):
    """(q, k, alpha, beta) = prep(...) with q_raw given, differentiable in the
    raw inputs (the gradients come from prep_bwd)."""
    return _Prepare.apply(q_raw, k_raw, a_raw, b_raw, bool(normalize_q), float(norm_eps))


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, h0, cu_seqlens, scale):
        o, hT = linear_fwd(q, k, v, g, h0, cu_seqlens, scale=scale)
        ctx.save_for_backward(q, k, v, g, h0, cu_seqlens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, hT

    @staticmethod
    @_once
    def backward(ctx, do, dhT):
        q, k, v, g, h0, cu = ctx.saved_tensors
        do = torch.zeros_like(v) if do is None else do.contiguous()
        dhT = None if dhT is None else dhT.contiguous()
        dq, dk, dv, dg, dh0 = linear_bwd(q, k, v, g, do, h0=h0, dhT=dhT, cu_seqlens=cu,
                                         scale=ctx.scale, store_dh0=h0 is not None)
        return dq, dk, dv, dg, dh0, None, None


def linear_attention(q, k, v, g, h0=None, cu_seqlens=None, scale=1.0):
    """(o, hT) = linear_fwd(...), differentiable in q, k, v, g and h0 (the
    gradients come from linear_bwd)."""
    return _LinearAttention.apply(q, k, v, g, h0, cu_seqlens, float(scale))


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layernorm_fwd(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        need = (weight is not None and ctx.needs_input_grad[1]) or \
            (ctx.has_bias and ctx.needs_input_grad[2])
        dx, dw, db = layernorm_bwd(dy.contiguous(), x, mean, rstd, weight, weight_grad=need)
        return dx, dw if weight is not None else None, db if ctx.has_bias else None, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """y = layernorm_fwd(...)[0], differentiable in x, weight and bias (the
    gradients come from layernorm_bwd).  A bias without a weight is fp32."""
    if weight is None and bias is not None and bias.dtype != torch.float32:
        raise TypeError(f"bias: dtype {bias.dtype}, expected {torch.float32} without a weight")
    return _LayerNorm.apply(x, weight, bias, float(eps))


def _or_zeros(grad, shape, like):
    if grad is None:
        return torch.zeros(shape, dtype=like.dtype, device=like.device)
    return grad.contiguous()


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, h0, cu_seqlens, silu):
        y, hT = conv_fwd(x, weight, bias, h0, cu_seqlens, silu)
        ctx.save_for_backward(x, weight, bias, h0, cu_seqlens)
        ctx.silu = silu
        ctx.set_materialize_grads(False)
        return y, hT

    @staticmethod
    @_once
    def backward(ctx, dy, dhT):
        x, weight, bias, h0, cu = ctx.saved_tensors
        dy = _or_zeros(dy, x.shape, x)
        dhT = None if dhT is None else dhT.contiguous()
        dx, dw, db, dh0 = conv_bwd(dy, x, weight, bias, h0=h0, dhT=dhT, cu_seqlens=cu, silu=ctx.silu,
                                   store_dh0=ctx.needs_input_grad[3])
        return dx, dw, db, dh0, None, None


def short_conv(x, weight, bias=None, h0=None, cu_seqlens=None, silu=True):
    """(y, hT) = conv_fwd(...), differentiable in x, weight, bias and h0 (the gradients come
    from conv_bwd)."""
    return _ShortConv.apply(x, weight, bias, h0, cu_seqlens, bool(silu))


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, softplus):
        y, hT = scan_fwd(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, softplus)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens)
        ctx.softplus = softplus
        ctx.set_materialize_grads(False)
        return y, hT

    @staticmethod
    @_once
    def backward(ctx, dy, dhT):
        x, dt, A, B, C, D, z, dt_bias, h0, cu = ctx.saved_tensors
        dy = _or_zeros(dy, x.shape, x)
        dhT = None if dhT is None else dhT.contiguous()
        return (*scan_bwd(dy, x, dt, A, B, C, D, z, dt_bias, h0, dhT, cu, ctx.softplus,
                          store_dh0=ctx.needs_input_grad[8]), None, None)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None,
                   softplus=True):
    """(y, hT) = scan_fwd(...), differentiable in x, dt, A, B, C, D, z, dt_bias and h0 (the
    gradients come from scan_bwd)."""
    return _SelectiveScan.apply(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, bool(softplus))


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = rmsnorm_fwd(x, weight, residual, eps=eps)
        ctx.save_for_backward(h, rstd, weight)
        ctx.added = residual is not None
        ctx.set_materialize_grads(False)
        return (y, h) if ctx.added else y

    @staticmethod
    @_once
    def backward(ctx, dy, dh=None):
        h, rstd, weight = ctx.saved_tensors
        dy = _or_zeros(dy, h.shape, h)
        dh = None if dh is None else dh.contiguous()
        dx, dw = rmsnorm_bwd(dy, h, rstd, weight, dh=dh,
                             weight_grad=weight is not None and ctx.needs_input_grad[1])
        return dx, dw, dx if ctx.added else None, None


def rms_norm(x, weight=None, residual=None, eps=1e-5):
    """y, or with a residual (y, h), of rmsnorm_fwd(...), differentiable in x, weight and
    residual (the gradients come from rmsnorm_bwd)."""
    return _RmsNorm.apply(x, weight, residual, float(eps))
