"""kda_chunkwise_b200 — Python binding of libkda (the KDA gated delta-rule recurrence on B200).

Argument marshalling only: every step of the recurrence runs in the CUDA kernels of libkda.so,
reached through its C ABI (include/kda.h).  PyTorch provides device memory and streams.  There is
no CPU or PyTorch fallback: importing this package without the built library raises ImportError.

Entry points (same names as the C ABI):
  kda_chunk_fwd(q, k, v, a, beta, A_log, cu_seqlens, ...)  prefill, chunkwise form
  kda_chunk_fwd_host(...)                                   the same prefill on host tensors, the copies
                                                            overlapped with the compute piece by piece
  kda_decode_step(q, k, v, a, beta, A_log, state, ...)      one recurrent step, state in place
  kda_decode_verify / kda_decode_commit                     K proposed tokens, then the accepted prefix
  kda_short_conv, kda_output_norm_gate                      the module's short convolution and
                                                            pre-gate normalisation + output gate
  kda_segment_maps, kda_state_combine,                      context-parallel prefill: a sequence split
  kda_context_parallel_fwd                                  into segments over the ranks of a group
  kda_chunk_bwd                                             gradients of the prefill (chunkwise=True: the
                                                            chunkwise form, kda_chunk_bwd_chunkwise)
  chunk_kda(...)                                            the prefill as a torch.autograd function: its
                                                            forward is kda_chunk_fwd, its backward kda_chunk_bwd
  kda_selective_scan_fwd / _step / _bwd, selective_scan     a state-space layer's scan: prompts, single tokens,
                                                            gradients, and as an autograd function
  kda_short_conv_fwd / _step / _bwd, short_conv             the short convolution with its carried window
  kda_layer_norm_fwd / _bwd, layer_norm                     layer norm
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

import torch

__all__ = ["kda_chunk_fwd", "kda_decode_step", "kda_chunk_fwd_workspace_size",
           "kda_chunk_fwd_workspace_min", "kda_sync_check", "kda_status_string", "KDAError",
           "kda_launch_count", "kda_chunk_fwd_noalloc", "kda_inject_stall",
           "kda_decode_verify", "kda_decode_commit", "kda_short_conv", "kda_output_norm_gate",
           "kda_state_combine", "kda_segment_maps", "context_parallel_states", "kda_context_parallel_fwd",
           "kda_chunk_bwd", "kda_chunk_bwd_workspace_size", "kda_chunk_fwd_host",
           "kda_chunk_fwd_host_buffer_size", "chunk_kda",
           "kda_selective_scan_fwd", "kda_selective_scan_fwd_workspace_size", "kda_selective_scan_step",
           "kda_selective_scan_bwd", "kda_selective_scan_bwd_workspace_size", "selective_scan",
           "kda_short_conv_fwd", "kda_short_conv_step", "kda_short_conv_bwd", "kda_short_conv_bwd_workspace_size",
           "short_conv", "kda_layer_norm_fwd", "kda_layer_norm_bwd", "kda_layer_norm_bwd_workspace_size",
           "layer_norm",
           "LIB_PATH", "lib"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_RANGE = range(6)
KDA_DTYPE_BF16, KDA_DTYPE_F32 = 0, 1
_OUT_DTYPES = {torch.bfloat16: KDA_DTYPE_BF16, torch.float32: KDA_DTYPE_F32}


class KDAError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {kda_status_string(status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libkda.so is not built ({LIB_PATH}); run `python "
                          "kda_chunkwise_b200/csrc/build.py` (nvcc 12.9, sm_100a) first")
    L = ctypes.CDLL(LIB_PATH)
    vp, fp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                 ctypes.c_int64, ctypes.c_size_t, ctypes.c_float)
    L.kda_chunk_fwd.argtypes = [vp, vp, vp, vp, fp, vp, fp, vp, i32, i64, i32, i32, i32, i32, f32,
                                fp, fp, vp, ctypes.c_int, vp, sz, vp]
    L.kda_chunk_fwd.restype = ctypes.c_int
    L.kda_chunk_fwd_noalloc.argtypes = [vp, vp, vp, vp, fp, vp, fp, vp, i32, i64, i32, i32, i32,
                                        i32, f32, fp, fp, vp, ctypes.c_int, vp]
    L.kda_chunk_fwd_noalloc.restype = ctypes.c_int
    L.kda_chunk_fwd_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32]
    L.kda_chunk_fwd_workspace_size.restype = sz
    L.kda_chunk_fwd_workspace_min.argtypes = [i64, i32, i32, i32, i32, i32]
    L.kda_chunk_fwd_workspace_min.restype = sz
    L.kda_decode_step.argtypes = [vp, vp, vp, vp, fp, vp, fp, fp, vp, ctypes.c_int, i32, i32, i32,
                                  i32, f32, vp]
    L.kda_decode_step.restype = ctypes.c_int
    L.kda_status_string.argtypes = [ctypes.c_int]
    L.kda_status_string.restype = ctypes.c_char_p
    L.kda_sync_check.argtypes = [vp]
    L.kda_sync_check.restype = ctypes.c_int
    L.kda_last_error.argtypes = []
    L.kda_last_error.restype = ctypes.c_char_p
    L.kda_launch_count.argtypes = []
    L.kda_launch_count.restype = ctypes.c_uint64
    L.kda_decode_verify.argtypes = [vp, vp, vp, vp, fp, vp, fp, fp, fp, vp, ctypes.c_int, i32, i32, i32,
                                    i32, i32, f32, vp]
    L.kda_decode_verify.restype = ctypes.c_int
    L.kda_decode_commit.argtypes = [vp, vp, fp, vp, fp, fp, i32, i32, i32, i32, i32, vp]
    L.kda_decode_commit.restype = ctypes.c_int
    L.kda_short_conv.argtypes = [vp, fp, vp, i32, i64, i32, i32, i32, i32, vp, vp]
    L.kda_short_conv.restype = ctypes.c_int
    L.kda_output_norm_gate.argtypes = [fp, vp, fp, i64, i32, i32, f32, vp, ctypes.c_int, vp]
    L.kda_output_norm_gate.restype = ctypes.c_int
    L.kda_state_combine.argtypes = [fp, fp, fp, fp, i32, i32, i32, vp]
    L.kda_state_combine.restype = ctypes.c_int
    L.kda_chunk_bwd.argtypes = [vp, vp, vp, vp, fp, vp, fp, vp, i32, i64, i32, i32, i32, f32, fp, fp, fp,
                                fp, fp, fp, fp, fp, fp, fp, fp, vp, sz, vp]
    L.kda_chunk_bwd.restype = ctypes.c_int
    L.kda_chunk_bwd_workspace_size.argtypes = [i64, i32, i32, i32, i32]
    L.kda_chunk_bwd_workspace_size.restype = sz
    L.kda_chunk_bwd_chunkwise.argtypes = L.kda_chunk_bwd.argtypes
    L.kda_chunk_bwd_chunkwise.restype = ctypes.c_int
    L.kda_chunk_bwd_chunkwise_workspace_size.argtypes = [i64, i32, i32, i32, i32]
    L.kda_chunk_bwd_chunkwise_workspace_size.restype = sz
    L.kda_chunk_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, f32, vp, vp, vp,
                                     ctypes.c_int, i64, vp, sz, vp]
    L.kda_chunk_fwd_host.restype = ctypes.c_int
    L.kda_chunk_fwd_host_buffer_size.argtypes = [vp, i32, i64, i32, i32, i32, ctypes.c_int, i64]
    L.kda_chunk_fwd_host_buffer_size.restype = sz
    L.kda_inject_stall.argtypes = [i32, ctypes.c_uint64]
    L.kda_inject_stall.restype = ctypes.c_int
    L.kda_set_prefill_path.argtypes = [i32]
    L.kda_set_prefill_path.restype = ctypes.c_int
    L.kda_prefill_path.argtypes = [i64, i32, i32]
    L.kda_prefill_path.restype = i32
    L.kda_segment_maps.argtypes = [vp, vp, vp, vp, fp, fp, vp, i32, i64, i32, i32, i32, f32, fp, fp, vp, sz, vp]
    L.kda_segment_maps.restype = ctypes.c_int
    L.kda_segment_maps_workspace_size.argtypes = [i64, i32, i32, i32]
    L.kda_segment_maps_workspace_size.restype = sz
    dtype = ctypes.c_int
    L.kda_selective_scan_fwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, vp, i32, i64, i32, i32, i32, fp, fp, vp,
                                         dtype, vp, sz, vp]
    L.kda_selective_scan_fwd.restype = ctypes.c_int
    L.kda_selective_scan_fwd_workspace_size.argtypes = [i64, i32, i32, i32, i32]
    L.kda_selective_scan_fwd_workspace_size.restype = sz
    L.kda_selective_scan_step.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, fp, vp, dtype, i32, i32, i32, i32, vp]
    L.kda_selective_scan_step.restype = ctypes.c_int
    L.kda_selective_scan_bwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, vp, i32, i64, i32, i32, i32, fp, vp, fp,
                                         vp, vp, fp, vp, vp, fp, vp, fp, fp, dtype, vp, sz, vp]
    L.kda_selective_scan_bwd.restype = ctypes.c_int
    L.kda_selective_scan_bwd_workspace_size.argtypes = [i64, i32, i32, i32, i32]
    L.kda_selective_scan_bwd_workspace_size.restype = sz
    L.kda_short_conv_fwd.argtypes = [vp, fp, fp, vp, i32, i64, i32, i32, i32, i32, i32, vp, vp, vp, dtype, vp]
    L.kda_short_conv_fwd.restype = ctypes.c_int
    L.kda_short_conv_step.argtypes = [vp, fp, fp, vp, i32, i32, i32, i32, i32, i32, vp, dtype, vp]
    L.kda_short_conv_step.restype = ctypes.c_int
    L.kda_short_conv_bwd.argtypes = [vp, fp, fp, vp, i32, i64, i32, i32, i32, i32, i32, vp, vp, vp, vp, fp, fp, vp,
                                     dtype, vp, sz, vp]
    L.kda_short_conv_bwd.restype = ctypes.c_int
    L.kda_short_conv_bwd_workspace_size.argtypes = [i64, i32, i32, i32]
    L.kda_short_conv_bwd_workspace_size.restype = sz
    L.kda_layer_norm_fwd.argtypes = [vp, fp, fp, i64, i32, f32, vp, fp, fp, dtype, vp]
    L.kda_layer_norm_fwd.restype = ctypes.c_int
    L.kda_layer_norm_bwd.argtypes = [vp, fp, fp, fp, vp, i64, i32, vp, fp, fp, dtype, vp, sz, vp]
    L.kda_layer_norm_bwd.restype = ctypes.c_int
    L.kda_layer_norm_bwd_workspace_size.argtypes = [i64, i32]
    L.kda_layer_norm_bwd_workspace_size.restype = sz
    return L


lib = _load()


def kda_status_string(status: int) -> str:
    return lib.kda_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != KDA_OK:
        raise KDAError(status, where, lib.kda_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype, shape, device):
    if t is not None and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def kda_chunk_fwd_workspace_size(total_tokens, num_seqs, max_seqlen, H, d_k, d_v) -> int:
    return int(lib.kda_chunk_fwd_workspace_size(total_tokens, num_seqs, max_seqlen, H, d_k, d_v))


def kda_chunk_fwd_workspace_min(total_tokens, num_seqs, max_seqlen, H, d_k, d_v) -> int:
    return int(lib.kda_chunk_fwd_workspace_min(total_tokens, num_seqs, max_seqlen, H, d_k, d_v))


def kda_chunk_fwd(q, k, v, a, beta, A_log, cu_seqlens, gate=None, initial_state=None,
                  output_final_state: bool = True, scale: float = 1.0, max_seqlen: int | None = None,
                  out=None, final_state=None, workspace=None, stream=None,
                  out_dtype=torch.bfloat16):
    """Chunkwise prefill over packed sequences (see include/kda.h for the full contract).

    q, k, a [T, H, d_k] bf16; v, gate [T, H, d_v] bf16; beta [T, H] fp32; A_log [H] fp32;
    cu_seqlens [N+1] int32 (device); initial_state [N, H, d_k, d_v] fp32 or None.
    max_seqlen: longest sequence (None: computed from cu_seqlens with one device->host copy).
    out_dtype: storage of the output, torch.bfloat16 or torch.float32 (taken from ``out`` if given).
    Returns (out [T, H, d_v], final_state [N, H, d_k, d_v] fp32 or None).
    """
    dev = q.device
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    N = cu_seqlens.numel() - 1
    bf = torch.bfloat16
    for name, t, shp in (("q", q, (T, H, d_k)), ("k", k, (T, H, d_k)), ("a", a, (T, H, d_k)),
                         ("v", v, (T, H, d_v))):
        _need(t, name, bf, shp, dev)
    _need(beta, "beta", torch.float32, (T, H), dev)
    _need(A_log, "A_log", torch.float32, (H,), dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    if gate is not None:
        _need(gate, "gate", bf, (T, H, d_v), dev)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (N, H, d_k, d_v), dev)
    if out is None:
        out = torch.empty((T, H, d_v), dtype=out_dtype, device=dev)
    if out.dtype not in _OUT_DTYPES:
        raise TypeError("out must be bfloat16 or float32")
    _need(out, "out", out.dtype, (T, H, d_v), dev)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, H, d_k, d_v), dtype=torch.float32, device=dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, (N, H, d_k, d_v), dev)
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if N > 0 else 0
    if workspace is None:
        nbytes = kda_chunk_fwd_workspace_size(T, N, max_seqlen, H, d_k, d_v)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    st = lib.kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(beta), _ptr(gate),
                           _ptr(A_log), _ptr(cu_seqlens), N, T, int(max_seqlen), H, d_k, d_v,
                           float(scale), _ptr(initial_state), _ptr(final_state), _ptr(out),
                           _OUT_DTYPES[out.dtype], _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream_handle(stream, dev))
    _check(st, "kda_chunk_fwd")
    return out, final_state


def kda_chunk_fwd_host_buffer_size(cu_seqlens, H, d_k, d_v, out_dtype=torch.bfloat16, piece_tokens: int = 0) -> int:
    """Device bytes kda_chunk_fwd_host needs; cu_seqlens is a host int32 tensor."""
    N = cu_seqlens.numel() - 1
    T = int(cu_seqlens[-1]) if N >= 0 else 0
    return int(lib.kda_chunk_fwd_host_buffer_size(_ptr(cu_seqlens), N, T, H, d_k, d_v, _OUT_DTYPES[out_dtype],
                                                  int(piece_tokens)))


def kda_chunk_fwd_host(q, k, v, a, beta, A_log, cu_seqlens, gate=None, initial_state=None, out=None,
                       final_state=None, out_dtype=torch.bfloat16, scale: float = 1.0, piece_tokens: int = 0,
                       device_buffer=None, device=None, stream=None):
    """Prefill of a batch held in host memory (see include/kda.h): every tensor, A_log and cu_seqlens
    included, is on the CPU (page-locked tensors let the copies overlap the compute).  The outputs
    ``out`` and ``final_state`` (host tensors; allocated page-locked when not given) hold the result
    once ``stream`` has reached the end of the call.  device_buffer: a CUDA uint8 tensor of
    kda_chunk_fwd_host_buffer_size(...) bytes (allocated when not given).
    Returns (out, final_state)."""
    cpu = torch.device("cpu")
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    N = cu_seqlens.numel() - 1
    bf = torch.bfloat16
    for name, t, shp in (("q", q, (T, H, d_k)), ("k", k, (T, H, d_k)), ("a", a, (T, H, d_k)),
                         ("v", v, (T, H, d_v))):
        _need(t, name, bf, shp, cpu)
    _need(beta, "beta", torch.float32, (T, H), cpu)
    _need(A_log, "A_log", torch.float32, (H,), cpu)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), cpu)
    if gate is not None:
        _need(gate, "gate", bf, (T, H, d_v), cpu)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (N, H, d_k, d_v), cpu)
    for name, t in (("q", q), ("k", k), ("a", a), ("v", v), ("beta", beta), ("gate", gate),
                    ("initial_state", initial_state), ("A_log", A_log), ("cu_seqlens", cu_seqlens)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out is None:
        out = torch.empty((T, H, d_v), dtype=out_dtype, pin_memory=True)
    if out.dtype not in _OUT_DTYPES:
        raise TypeError("out must be bfloat16 or float32")
    _need(out, "out", out.dtype, (T, H, d_v), cpu)
    if final_state is None:
        final_state = torch.empty((N, H, d_k, d_v), dtype=torch.float32, pin_memory=True)
    _need(final_state, "final_state", torch.float32, (N, H, d_k, d_v), cpu)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device_buffer is None:
        nbytes = kda_chunk_fwd_host_buffer_size(cu_seqlens, H, d_k, d_v, out.dtype, piece_tokens)
        device_buffer = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    st = lib.kda_chunk_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(beta), _ptr(gate), _ptr(A_log),
                                _ptr(cu_seqlens), N, T, H, d_k, d_v, float(scale), _ptr(initial_state),
                                _ptr(final_state), _ptr(out), _OUT_DTYPES[out.dtype], int(piece_tokens),
                                _ptr(device_buffer), device_buffer.numel(), _stream_handle(stream, dev))
    _check(st, "kda_chunk_fwd_host")
    return out, final_state


def kda_chunk_fwd_noalloc(q, k, v, a, beta, A_log, cu_seqlens, max_seqlen: int, gate=None,
                          initial_state=None, scale: float = 1.0, out=None, final_state=None,
                          stream=None):
    """kda_chunk_fwd on the library's built-in 32 MiB scratch instead of a workspace.

    For callers that cannot allocate device memory on this path: it allocates nothing (the
    caller passes ``out`` and ``final_state`` if it wants them; ``out`` is required and its dtype,
    bfloat16 or float32, selects the output storage).  Calls on one device share the scratch:
    keep them on one stream.  max_seqlen must be given (no device-to-host read is made).
    """
    dev = q.device
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    N = cu_seqlens.numel() - 1
    bf = torch.bfloat16
    for name, t, shp in (("q", q, (T, H, d_k)), ("k", k, (T, H, d_k)), ("a", a, (T, H, d_k)),
                         ("v", v, (T, H, d_v))):
        _need(t, name, bf, shp, dev)
    _need(beta, "beta", torch.float32, (T, H), dev)
    _need(A_log, "A_log", torch.float32, (H,), dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    if gate is not None:
        _need(gate, "gate", bf, (T, H, d_v), dev)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (N, H, d_k, d_v), dev)
    if out is None or out.dtype not in _OUT_DTYPES:
        raise ValueError("out (bfloat16 or float32, [T, H, d_v]) is required")
    _need(out, "out", out.dtype, (T, H, d_v), dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, (N, H, d_k, d_v), dev)
    st = lib.kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(beta), _ptr(gate),
                                   _ptr(A_log), _ptr(cu_seqlens), N, T, int(max_seqlen), H, d_k,
                                   d_v, float(scale), _ptr(initial_state), _ptr(final_state),
                                   _ptr(out), _OUT_DTYPES[out.dtype], _stream_handle(stream, dev))
    _check(st, "kda_chunk_fwd_noalloc")
    return out, final_state


def kda_decode_step(q, k, v, a, beta, A_log, state, gate=None, scale: float = 1.0, out=None,
                    stream=None, out_dtype=torch.bfloat16):
    """One recurrent step for N sequences; ``state`` [N, H, d_k, d_v] fp32 is updated in place.

    q, k, a [N, H, d_k] bf16; v, gate [N, H, d_v] bf16; beta [N, H] fp32; A_log [H] fp32.
    Returns out [N, H, d_v] (bfloat16 or float32, see kda_chunk_fwd).
    """
    dev = q.device
    N, H, d_k = q.shape
    d_v = v.shape[-1]
    bf = torch.bfloat16
    for name, t, shp in (("q", q, (N, H, d_k)), ("k", k, (N, H, d_k)), ("a", a, (N, H, d_k)),
                         ("v", v, (N, H, d_v))):
        _need(t, name, bf, shp, dev)
    _need(beta, "beta", torch.float32, (N, H), dev)
    _need(A_log, "A_log", torch.float32, (H,), dev)
    _need(state, "state", torch.float32, (N, H, d_k, d_v), dev)
    if gate is not None:
        _need(gate, "gate", bf, (N, H, d_v), dev)
    if out is None:
        out = torch.empty((N, H, d_v), dtype=out_dtype, device=dev)
    if out.dtype not in _OUT_DTYPES:
        raise TypeError("out must be bfloat16 or float32")
    _need(out, "out", out.dtype, (N, H, d_v), dev)
    st = lib.kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(beta), _ptr(gate),
                             _ptr(A_log), _ptr(state), _ptr(out), _OUT_DTYPES[out.dtype], N, H,
                             d_k, d_v, float(scale),
                             _stream_handle(stream, dev))
    _check(st, "kda_decode_step")
    return out


def kda_decode_verify(q, k, v, a, beta, A_log, state, gate=None, scale: float = 1.0, u=None, out=None,
                      stream=None, out_dtype=torch.bfloat16):
    """Run K proposed tokens of N sequences from ``state`` without changing it.

    q, k, a [N, K, H, d_k] bf16; v, gate [N, K, H, d_v] bf16; beta [N, K, H] fp32; A_log [H];
    state [N, H, d_k, d_v] fp32 (read only).  Returns (out [N, K, H, d_v], u [N, H, K, d_v] fp32);
    pass u to kda_decode_commit.
    """
    dev = q.device
    N, K, H, d_k = q.shape
    d_v = v.shape[-1]
    bf = torch.bfloat16
    for name, t, shp in (("q", q, (N, K, H, d_k)), ("k", k, (N, K, H, d_k)), ("a", a, (N, K, H, d_k)),
                         ("v", v, (N, K, H, d_v))):
        _need(t, name, bf, shp, dev)
    _need(beta, "beta", torch.float32, (N, K, H), dev)
    _need(A_log, "A_log", torch.float32, (H,), dev)
    _need(state, "state", torch.float32, (N, H, d_k, d_v), dev)
    if gate is not None:
        _need(gate, "gate", bf, (N, K, H, d_v), dev)
    if u is None:
        u = torch.empty((N, H, K, d_v), dtype=torch.float32, device=dev)
    _need(u, "u", torch.float32, (N, H, K, d_v), dev)
    if out is None:
        out = torch.empty((N, K, H, d_v), dtype=out_dtype, device=dev)
    if out.dtype not in _OUT_DTYPES:
        raise TypeError("out must be bfloat16 or float32")
    _need(out, "out", out.dtype, (N, K, H, d_v), dev)
    st = lib.kda_decode_verify(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(beta), _ptr(gate), _ptr(A_log),
                               _ptr(state), _ptr(u), _ptr(out), _OUT_DTYPES[out.dtype], N, K, H, d_k, d_v,
                               float(scale), _stream_handle(stream, dev))
    _check(st, "kda_decode_verify")
    return out, u


def kda_decode_commit(k, a, A_log, accepted, u, state, stream=None):
    """Advance each state by its accepted[n] verified tokens (int32 [N] on the device); in place."""
    dev = k.device
    N, K, H, d_k = k.shape
    d_v = u.shape[-1]
    _need(k, "k", torch.bfloat16, (N, K, H, d_k), dev)
    _need(a, "a", torch.bfloat16, (N, K, H, d_k), dev)
    _need(A_log, "A_log", torch.float32, (H,), dev)
    _need(accepted, "accepted", torch.int32, (N,), dev)
    _need(u, "u", torch.float32, (N, H, K, d_v), dev)
    _need(state, "state", torch.float32, (N, H, d_k, d_v), dev)
    st = lib.kda_decode_commit(_ptr(k), _ptr(a), _ptr(A_log), _ptr(accepted), _ptr(u), _ptr(state),
                               N, K, H, d_k, d_v, _stream_handle(stream, dev))
    _check(st, "kda_decode_commit")
    return state


def kda_short_conv(x, w, cu_seqlens, l2norm: bool = False, out=None, stream=None):
    """Causal depthwise convolution over time per packed sequence (bf16 [T, H, d] in and out),
    optionally L2-normalising every (token, head) row.  w: fp32 [H, d, width], width <= 4."""
    dev = x.device
    T, H, d = x.shape
    width = w.shape[-1]
    _need(x, "x", torch.bfloat16, (T, H, d), dev)
    _need(w, "w", torch.float32, (H, d, width), dev)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != dev or cu_seqlens.dim() != 1:
        raise TypeError("cu_seqlens must be int32 [num_seqs + 1] on the device")
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", torch.bfloat16, (T, H, d), dev)
    st = lib.kda_short_conv(_ptr(x), _ptr(w), _ptr(cu_seqlens), cu_seqlens.numel() - 1, T, H, d, width,
                            1 if l2norm else 0, _ptr(out), _stream_handle(stream, dev))
    _check(st, "kda_short_conv")
    return out


def kda_output_norm_gate(o, gate, w, eps: float = 1e-6, out=None, stream=None, out_dtype=torch.bfloat16):
    """out = sigmoid(gate) * RMSNorm(o) * w per (token, head) row; o fp32 [T, H, d_v], gate bf16 or
    None, w fp32 [d_v]."""
    dev = o.device
    T, H, d_v = o.shape
    _need(o, "o", torch.float32, (T, H, d_v), dev)
    _need(w, "w", torch.float32, (d_v,), dev)
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, (T, H, d_v), dev)
    if out is None:
        out = torch.empty((T, H, d_v), dtype=out_dtype, device=dev)
    if out.dtype not in _OUT_DTYPES:
        raise TypeError("out must be bfloat16 or float32")
    _need(out, "out", out.dtype, (T, H, d_v), dev)
    st = lib.kda_output_norm_gate(_ptr(o), _ptr(gate), _ptr(w), T, H, d_v, float(eps), _ptr(out),
                                  _OUT_DTYPES[out.dtype], _stream_handle(stream, dev))
    _check(st, "kda_output_norm_gate")
    return out


def kda_state_combine(M, S_in, B, out=None, stream=None):
    """S_out = M S_in + B per (sequence, head): M fp32 [..., d_k, d_k], S_in and B [..., d_k, d_v]."""
    dev = M.device
    d_k, d_v = B.shape[-2], B.shape[-1]
    lead = tuple(B.shape[:-2])
    units = int(np.prod(lead)) if lead else 1
    _need(M, "M", torch.float32, lead + (d_k, d_k), dev)
    _need(S_in, "S_in", torch.float32, lead + (d_k, d_v), dev)
    _need(B, "B", torch.float32, lead + (d_k, d_v), dev)
    if out is None:
        out = torch.empty_like(B)
    _need(out, "out", torch.float32, lead + (d_k, d_v), dev)
    st = lib.kda_state_combine(_ptr(M), _ptr(S_in), _ptr(B), _ptr(out), units, d_k, d_v,
                               _stream_handle(stream, dev))
    _check(st, "kda_state_combine")
    return out


def kda_segment_maps(q, k, v, a, beta, A_log, cu_seqlens, scale: float = 1.0, max_seqlen=None, stream=None,
                     single_pass: bool | None = None):
    """The affine map S -> M S + B of each (sequence, head) over the tokens given: B is the final
    state from S = 0, M the final state of the homogeneous recurrence (v = 0) from S = I.  Returns
    (M [N, H, d_k, d_k], B [N, H, d_k, d_v]).

    single_pass: one pass of the cluster kernel over value columns [0 | v] from [I | 0]
    (kda_segment_maps; d_k = d_v only), which shares the chunk-local work of both maps but needs
    2 d / 32 CTAs per unit; or two kda_chunk_fwd calls.  None: one pass when every unit's cluster
    fits the GPU at once (then it takes the time of one of the two calls), else two calls (the same
    SM time, and with many units kda_chunk_fwd's per-unit kernel is the faster one)."""
    N = cu_seqlens.numel() - 1
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    dev = q.device
    if single_pass is None:
        sms = torch.cuda.get_device_properties(dev).multi_processor_count if dev.type == "cuda" else 0
        single_pass = N * H * (2 * d_k // 32) <= sms
    if single_pass and d_k == d_v:
        for name, t in (("q", q), ("k", k), ("v", v), ("a", a)):
            _need(t, name, torch.bfloat16, (T, H, d_k), dev)
        _need(beta, "beta", torch.float32, (T, H), dev)
        _need(A_log, "A_log", torch.float32, (H,), dev)
        _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
        if max_seqlen is None:
            max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if N > 0 else 0
        M = torch.empty((N, H, d_k, d_k), dtype=torch.float32, device=dev)
        B = torch.empty((N, H, d_k, d_k), dtype=torch.float32, device=dev)
        ws = torch.empty(max(int(lib.kda_segment_maps_workspace_size(T, N, H, d_k)), 1), dtype=torch.uint8, device=dev)
        st = lib.kda_segment_maps(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(beta), _ptr(A_log), _ptr(cu_seqlens), N, T,
                                  max_seqlen, H, d_k, scale, _ptr(M), _ptr(B), _ptr(ws), ws.numel(),
                                  _stream_handle(stream, dev))
        _check(st, "kda_segment_maps")
        return M, B
    _, B = kda_chunk_fwd(q, k, v, a, beta, A_log, cu_seqlens, gate=None, initial_state=None, scale=scale,
                         max_seqlen=max_seqlen, stream=stream, out_dtype=torch.bfloat16)
    v0 = torch.zeros((T, H, d_k), dtype=torch.bfloat16, device=q.device)
    eye = torch.eye(d_k, dtype=torch.float32, device=q.device).expand(N, H, d_k, d_k).contiguous()
    _, M = kda_chunk_fwd(q, k, v0, a, beta, A_log, cu_seqlens, gate=None, initial_state=eye, scale=scale,
                         max_seqlen=max_seqlen, stream=stream, out_dtype=torch.bfloat16)
    return M, B


def context_parallel_states(M, B, S0, group=None, combine=None):
    """Incoming state of this rank's segments: gather every rank's (M, B) over the process group and
    fold the maps of the ranks before this one, in rank order, starting from S0.  ``combine(M, S, B)``
    applies one map (kda_state_combine unless given)."""
    import torch.distributed as dist
    combine = combine or (lambda m, s, b: kda_state_combine(m, s, b))
    world = dist.get_world_size(group) if dist.is_available() and dist.is_initialized() else 1
    S = S0.clone() if S0 is not None else torch.zeros_like(B)
    if world == 1:
        return S
    rank = dist.get_rank(group)

    # NCCL gathers device tensors directly; gloo (CPU ranks, or ranks sharing one GPU) goes through
    # host copies
    via_host = M.is_cuda and dist.get_backend(group) == "gloo"

    def gather(x):   # every rank's x, stacked in rank order
        src = x.contiguous().cpu() if via_host else x.contiguous()
        flat = torch.empty((world * src.shape[0],) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
        dist.all_gather_into_tensor(flat, src, group=group)
        flat = flat.to(x.device) if via_host else flat
        return flat.view((world,) + tuple(x.shape))

    Ms, Bs = gather(M), gather(B)
    for r in range(rank):
        S = combine(Ms[r], S, Bs[r])
    return S


def kda_context_parallel_fwd(q, k, v, a, beta, A_log, cu_seqlens, gate=None, initial_state=None,
                             scale: float = 1.0, group=None, max_seqlen=None, stream=None,
                             out_dtype=torch.bfloat16):
    """Prefill of sequences split along time over the ranks of ``group``: this rank holds segment
    `rank` of every sequence (the same sequences, in the same order, on every rank; segments in
    rank order).  ``initial_state`` is the sequences' initial state (the same on every rank).
    Returns (out of this segment, state after this segment): on the last rank, the final states."""
    M, B = kda_segment_maps(q, k, v, a, beta, A_log, cu_seqlens, scale=scale, max_seqlen=max_seqlen,
                            stream=stream)
    S_in = context_parallel_states(M, B, initial_state, group=group)
    return kda_chunk_fwd(q, k, v, a, beta, A_log, cu_seqlens, gate=gate, initial_state=S_in, scale=scale,
                         max_seqlen=max_seqlen, stream=stream, out_dtype=out_dtype)


def kda_chunk_bwd_workspace_size(total_tokens, num_seqs, H, d_k, d_v) -> int:
    return int(lib.kda_chunk_bwd_workspace_size(total_tokens, num_seqs, H, d_k, d_v))


def kda_chunk_bwd_chunkwise_workspace_size(total_tokens, num_seqs, H, d_k, d_v) -> int:
    return int(lib.kda_chunk_bwd_chunkwise_workspace_size(total_tokens, num_seqs, H, d_k, d_v))


def kda_chunk_bwd(q, k, v, a, beta, A_log, cu_seqlens, dout, gate=None, initial_state=None,
                  dfinal_state=None, scale: float = 1.0, workspace=None, stream=None, chunkwise: bool = False):
    """Gradients of kda_chunk_fwd's outputs (and final states) with respect to its inputs.

    dout fp32 [T, H, d_v]; dfinal_state fp32 [N, H, d_k, d_v] or None.  Returns a dict of fp32
    tensors: dq, dk, da [T, H, d_k]; dv, dgate [T, H, d_v] (dgate None without a gate); dbeta
    [T, H]; dA_log [H]; dinitial_state [N, H, d_k, d_v] (None without an initial state).
    chunkwise: run kda_chunk_bwd_chunkwise (the chunkwise form) instead of the token-level kernel;
    the gradients agree to rounding.
    """
    dev = q.device
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    N = cu_seqlens.numel() - 1
    bf, f32 = torch.bfloat16, torch.float32
    for name, t, shp in (("q", q, (T, H, d_k)), ("k", k, (T, H, d_k)), ("a", a, (T, H, d_k)),
                         ("v", v, (T, H, d_v))):
        _need(t, name, bf, shp, dev)
    _need(beta, "beta", f32, (T, H), dev)
    _need(A_log, "A_log", f32, (H,), dev)
    _need(dout, "dout", f32, (T, H, d_v), dev)
    if gate is not None:
        _need(gate, "gate", bf, (T, H, d_v), dev)
    if initial_state is not None:
        _need(initial_state, "initial_state", f32, (N, H, d_k, d_v), dev)
    if dfinal_state is not None:
        _need(dfinal_state, "dfinal_state", f32, (N, H, d_k, d_v), dev)
    g = dict(dq=torch.empty((T, H, d_k), dtype=f32, device=dev), dk=torch.empty((T, H, d_k), dtype=f32, device=dev),
             da=torch.empty((T, H, d_k), dtype=f32, device=dev), dv=torch.empty((T, H, d_v), dtype=f32, device=dev),
             dbeta=torch.empty((T, H), dtype=f32, device=dev), dA_log=torch.empty((H,), dtype=f32, device=dev),
             dgate=None if gate is None else torch.empty((T, H, d_v), dtype=f32, device=dev),
             dinitial_state=None if initial_state is None else torch.empty((N, H, d_k, d_v), dtype=f32, device=dev))
    need = (kda_chunk_bwd_chunkwise_workspace_size if chunkwise else kda_chunk_bwd_workspace_size)(T, N, H, d_k, d_v)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    fn = lib.kda_chunk_bwd_chunkwise if chunkwise else lib.kda_chunk_bwd
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(beta), _ptr(gate), _ptr(A_log),
                           _ptr(cu_seqlens), N, T, H, d_k, d_v, float(scale), _ptr(initial_state), _ptr(dout),
                           _ptr(dfinal_state), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["da"]),
                           _ptr(g["dbeta"]), _ptr(g["dgate"]), _ptr(g["dA_log"]), _ptr(g["dinitial_state"]),
                           _ptr(workspace), workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    _check(st, "kda_chunk_bwd_chunkwise" if chunkwise else "kda_chunk_bwd")
    return g


class _ChunkKDA(torch.autograd.Function):
    """kda_chunk_fwd forward, kda_chunk_bwd backward (both through the C ABI); the gradients come
    back in fp32 and are cast to each input's dtype."""

    @staticmethod
    def forward(ctx, q, k, v, a, beta, A_log, gate, initial_state, cu_seqlens, scale, out_dtype):
        out, S = kda_chunk_fwd(q, k, v, a, beta, A_log, cu_seqlens, gate=gate, initial_state=initial_state,
                               scale=scale, out_dtype=out_dtype)
        ctx.save_for_backward(q, k, v, a, beta, A_log, gate, initial_state, cu_seqlens)
        ctx.scale = scale
        return out, S

    @staticmethod
    def backward(ctx, dout, dS):
        q, k, v, a, beta, A_log, gate, initial_state, cu_seqlens = ctx.saved_tensors
        if dout is None:
            dout = torch.zeros((q.shape[0], q.shape[1], v.shape[-1]), dtype=torch.float32, device=q.device)
        g = kda_chunk_bwd(q, k, v, a, beta, A_log, cu_seqlens, dout.to(torch.float32).contiguous(), gate=gate,
                          initial_state=initial_state, dfinal_state=None if dS is None else dS.contiguous(),
                          scale=ctx.scale)
        like = lambda x, ref: None if x is None or ref is None else x.to(ref.dtype)
        return (like(g["dq"], q), like(g["dk"], k), like(g["dv"], v), like(g["da"], a), g["dbeta"], g["dA_log"],
                like(g["dgate"], gate), g["dinitial_state"], None, None, None)


def chunk_kda(q, k, v, a, beta, A_log, cu_seqlens, gate=None, initial_state=None, scale: float = 1.0,
              out_dtype=torch.bfloat16):
    """The prefill (kda_chunk_fwd) as a differentiable function of q, k, v, a, beta, A_log, gate and
    initial_state.  Returns (out [T, H, d_v], final_state [N, H, d_k, d_v] fp32); a loss on either
    or both reaches the inputs through kda_chunk_bwd."""
    return _ChunkKDA.apply(q, k, v, a, beta, A_log, gate, initial_state, cu_seqlens, float(scale), out_dtype)


# ---- the selective scan, the convolution with its carried window, layer norm ---------------------


class _Call:
    """Where a call's work runs: its device is made current, and what it allocates belongs to its stream."""

    __slots__ = ("device", "handle", "_with")

    def __init__(self, x, stream):
        if not x.is_cuda:
            raise ValueError(f"tensors must be on a CUDA device, got {x.device}")
        self.device, self._with = x.device, None
        index = x.get_device()
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(index)
        elif stream.device != x.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {x.device}")
        else:
            self.handle = stream.cuda_stream
        if stream is not None or index != torch.cuda.current_device():
            # (a stream's context makes its device current too)
            self._with = torch.cuda.device(x.device) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self._with is not None:
            self._with.__enter__()
        return self

    def __exit__(self, *exc):
        if self._with is not None:
            self._with.__exit__(*exc)

    def empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    @staticmethod
    def like(t):
        """An output of a checked (dense) tensor's shape and type; None for None."""
        return None if t is None else torch.empty_like(t)

    def workspace(self, given, nbytes):
        if given is None:
            return (torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None), nbytes
        if given.device != self.device or not given.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {self.device}")
        return given, given.numel() * given.element_size()


def _io_dtype(x, name):
    if x.dtype not in _OUT_DTYPES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {x.dtype}")
    return _OUT_DTYPES[x.dtype]


def _scan_args(u, dt, A_log, B, C, skip, z, dt_bias):
    """Checks what the scan's calls share; returns (rows, D, n, G, dtype code)."""
    code = _io_dtype(u, "u")
    if u.dim() != 2 or B.dim() != 3 or A_log.dim() != 2:
        raise ValueError("u must be [tokens, D], B [tokens, G, n] and A_log [D, n]")
    rows, D = u.shape
    G, n = B.shape[1:]
    dev, t, f32 = u.device, u.dtype, torch.float32
    _need(u, "u", t, (rows, D), dev)
    _need(dt, "dt", t, (rows, D), dev)
    _need(A_log, "A_log", f32, (D, n), dev)
    _need(B, "B", t, (rows, G, n), dev)
    _need(C, "C", t, (rows, G, n), dev)
    if z is not None:
        _need(z, "z", t, (rows, D), dev)
    if skip is not None:
        _need(skip, "skip", f32, (D,), dev)
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", f32, (D,), dev)
    return rows, D, n, G, code


def _need_seqlens(cu_seqlens, dev):
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be int32 [num_seqs + 1]")
    _need(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, dev)
    return cu_seqlens.numel() - 1


def kda_selective_scan_fwd_workspace_size(total_tokens, num_seqs, D, n, G=1) -> int:
    return int(lib.kda_selective_scan_fwd_workspace_size(total_tokens, num_seqs, D, n, G))


def kda_selective_scan_bwd_workspace_size(total_tokens, num_seqs, D, n, G=1) -> int:
    return int(lib.kda_selective_scan_bwd_workspace_size(total_tokens, num_seqs, D, n, G))


def kda_selective_scan_fwd(u, dt, A_log, B, C, cu_seqlens, skip=None, z=None, dt_bias=None, initial_state=None,
                           output_final_state: bool = True, out=None, final_state=None, workspace=None, stream=None):
    """Selective state space scan over packed sequences (see include/kda.h):
    h_t = exp(delta A) h_{t-1} + delta u B_t, out_t = silu(z) (C_t h_t + skip u), delta = softplus(dt + dt_bias),
    A = -exp(A_log).

    u, dt, z [T, D] and B, C [T, G, n], all bfloat16 or all float32; A_log fp32 [D, n]; skip, dt_bias fp32
    [D] or None; cu_seqlens int32 [N + 1] (device); initial_state fp32 [N, D, n] or None; final_state may
    be initial_state.  Returns (out [T, D], final_state fp32 [N, D, n] or None)."""
    T, D, n, G, code = _scan_args(u, dt, A_log, B, C, skip, z, dt_bias)
    N = _need_seqlens(cu_seqlens, u.device)
    f32 = torch.float32
    if initial_state is not None:
        _need(initial_state, "initial_state", f32, (N, D, n), u.device)
    with _Call(u, stream) as call:
        if out is None:
            out = call.like(u)
        _need(out, "out", u.dtype, (T, D), u.device)
        if final_state is None and output_final_state:
            final_state = call.empty((N, D, n), f32)
        if final_state is not None:
            _need(final_state, "final_state", f32, (N, D, n), u.device)
        ws, ws_bytes = call.workspace(workspace, kda_selective_scan_fwd_workspace_size(T, N, D, n, G))
        st = lib.kda_selective_scan_fwd(_ptr(u), _ptr(dt), _ptr(A_log), _ptr(B), _ptr(C), _ptr(skip), _ptr(z),
                                        _ptr(dt_bias), _ptr(cu_seqlens), N, T, D, n, G, _ptr(initial_state),
                                        _ptr(final_state), _ptr(out), code, _ptr(ws), ws_bytes, call.handle)
    _check(st, "kda_selective_scan_fwd")
    return out, final_state


def kda_selective_scan_step(u, dt, A_log, B, C, state, skip=None, z=None, dt_bias=None, out=None, stream=None):
    """One token of N sequences; ``state`` fp32 [N, D, n] is updated in place.  u, dt, z [N, D]; B, C
    [N, G, n]; the rest as kda_selective_scan_fwd.  Returns out [N, D]."""
    N, D, n, G, code = _scan_args(u, dt, A_log, B, C, skip, z, dt_bias)
    _need(state, "state", torch.float32, (N, D, n), u.device)
    with _Call(u, stream) as call:
        if out is None:
            out = call.like(u)
        else:
            _need(out, "out", u.dtype, (N, D), u.device)
        st = lib.kda_selective_scan_step(_ptr(u), _ptr(dt), _ptr(A_log), _ptr(B), _ptr(C), _ptr(skip), _ptr(z),
                                         _ptr(dt_bias), _ptr(state), _ptr(out), code, N, D, n, G, call.handle)
    _check(st, "kda_selective_scan_step")
    return out


def kda_selective_scan_bwd(u, dt, A_log, B, C, cu_seqlens, dout, skip=None, z=None, dt_bias=None, initial_state=None,
                           dfinal_state=None, workspace=None, stream=None):
    """Gradients of kda_selective_scan_fwd with the same inputs.  dout of u's dtype [T, D]; dfinal_state fp32
    [N, D, n] or None.  Returns a dict: du, ddt, dz [T, D] and dB, dC [T, G, n] of u's dtype; dA_log [D, n],
    dskip, ddt_bias [D], dinitial_state [N, D, n] fp32; None for what was not given."""
    T, D, n, G, code = _scan_args(u, dt, A_log, B, C, skip, z, dt_bias)
    N = _need_seqlens(cu_seqlens, u.device)
    f32, t, dev = torch.float32, u.dtype, u.device
    _need(dout, "dout", t, (T, D), dev)
    if initial_state is not None:
        _need(initial_state, "initial_state", f32, (N, D, n), dev)
    if dfinal_state is not None:
        _need(dfinal_state, "dfinal_state", f32, (N, D, n), dev)
    with _Call(u, stream) as call:
        g = dict(du=call.like(u), ddt=call.like(dt), dA_log=call.like(A_log), dB=call.like(B), dC=call.like(C),
                 dskip=call.like(skip), dz=call.like(z), ddt_bias=call.like(dt_bias),
                 dinitial_state=call.like(initial_state))
        ws, ws_bytes = call.workspace(workspace, kda_selective_scan_bwd_workspace_size(T, N, D, n, G))
        st = lib.kda_selective_scan_bwd(_ptr(u), _ptr(dt), _ptr(A_log), _ptr(B), _ptr(C), _ptr(skip), _ptr(z),
                                        _ptr(dt_bias), _ptr(cu_seqlens), N, T, D, n, G, _ptr(initial_state),
                                        _ptr(dout), _ptr(dfinal_state), _ptr(g["du"]), _ptr(g["ddt"]),
                                        _ptr(g["dA_log"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dskip"]),
                                        _ptr(g["dz"]), _ptr(g["ddt_bias"]), _ptr(g["dinitial_state"]), code, _ptr(ws),
                                        ws_bytes, call.handle)
    _check(st, "kda_selective_scan_bwd")
    return g


def _conv_args(x, w, bias):
    code = _io_dtype(x, "x")
    if x.dim() != 3 or w.dim() != 3:
        raise ValueError("x must be [tokens, H, d] and w [H, d, width]")
    rows, H, d = x.shape
    W = w.shape[2]
    _need(x, "x", x.dtype, (rows, H, d), x.device)
    _need(w, "w", torch.float32, (H, d, W), x.device)
    if bias is not None:
        _need(bias, "bias", torch.float32, (H, d), x.device)
    return rows, H, d, W, code


def kda_short_conv_fwd(x, w, cu_seqlens, bias=None, initial_state=None, silu: bool = False, l2norm: bool = False,
                       output_final_state: bool = True, out=None, final_state=None, stream=None):
    """Causal depthwise convolution over packed sequences with its carried window (see include/kda.h):
    bias + sum_j w[..., j] x_{t-(width-1)+j}, then SiLU, then L2 normalisation per head, each optional.

    x [T, H, d] bfloat16 or float32; w fp32 [H, d, width], width <= 4; bias fp32 [H, d] or None;
    initial_state [N, width - 1, H, d] of x's dtype or None: the inputs before each sequence, oldest first;
    final_state likewise (it may be initial_state).  Returns (y [T, H, d], final_state or None)."""
    T, H, d, W, code = _conv_args(x, w, bias)
    N = _need_seqlens(cu_seqlens, x.device)
    state = (N, W - 1, H, d)
    if initial_state is not None:
        _need(initial_state, "initial_state", x.dtype, state, x.device)
    with _Call(x, stream) as call:
        if out is None:
            out = call.like(x)
        _need(out, "out", x.dtype, (T, H, d), x.device)
        if final_state is None and output_final_state:
            final_state = call.empty(state, x.dtype)
        if final_state is not None:
            _need(final_state, "final_state", x.dtype, state, x.device)
        st = lib.kda_short_conv_fwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(cu_seqlens), N, T, H, d, W, int(silu), int(l2norm),
                                    _ptr(initial_state), _ptr(final_state), _ptr(out), code, call.handle)
    _check(st, "kda_short_conv_fwd")
    return out, final_state


def kda_short_conv_step(x, w, state, bias=None, silu: bool = False, l2norm: bool = False, out=None, stream=None):
    """One token of N sequences: x [N, H, d]; ``state`` [N, width - 1, H, d] of x's dtype is updated in
    place.  The rest as kda_short_conv_fwd.  Returns y [N, H, d]."""
    N, H, d, W, code = _conv_args(x, w, bias)
    _need(state, "state", x.dtype, (N, W - 1, H, d), x.device)
    with _Call(x, stream) as call:
        if out is None:
            out = call.like(x)
        else:
            _need(out, "out", x.dtype, (N, H, d), x.device)
        st = lib.kda_short_conv_step(_ptr(x), _ptr(w), _ptr(bias), _ptr(state), N, H, d, W, int(silu), int(l2norm),
                                     _ptr(out), code, call.handle)
    _check(st, "kda_short_conv_step")
    return out


def kda_short_conv_bwd_workspace_size(total_tokens, H, d, width) -> int:
    return int(lib.kda_short_conv_bwd_workspace_size(total_tokens, H, d, width))


def kda_short_conv_bwd(x, w, cu_seqlens, dy, bias=None, initial_state=None, dfinal_state=None, silu: bool = False,
                       l2norm: bool = False, workspace=None, stream=None):
    """Gradients of kda_short_conv_fwd with the same inputs; dy [T, H, d] and dfinal_state (or None) of x's
    dtype.  Returns a dict: dx and dinitial_state of x's dtype, dw [H, d, width] and dbias [H, d] fp32; None
    for what was not given."""
    T, H, d, W, code = _conv_args(x, w, bias)
    N = _need_seqlens(cu_seqlens, x.device)
    state, t = (N, W - 1, H, d), x.dtype
    _need(dy, "dy", t, (T, H, d), x.device)
    for name, s in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if s is not None:
            _need(s, name, t, state, x.device)
    with _Call(x, stream) as call:
        g = dict(dx=call.like(x), dw=call.like(w), dbias=call.like(bias), dinitial_state=call.like(initial_state))
        ws, ws_bytes = call.workspace(workspace, kda_short_conv_bwd_workspace_size(T, H, d, W))
        st = lib.kda_short_conv_bwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(cu_seqlens), N, T, H, d, W, int(silu), int(l2norm),
                                    _ptr(initial_state), _ptr(dy), _ptr(dfinal_state), _ptr(g["dx"]), _ptr(g["dw"]),
                                    _ptr(g["dbias"]), _ptr(g["dinitial_state"]), code, _ptr(ws), ws_bytes, call.handle)
    _check(st, "kda_short_conv_bwd")
    return g


def kda_layer_norm_bwd_workspace_size(rows, d) -> int:
    return int(lib.kda_layer_norm_bwd_workspace_size(rows, d))


def kda_layer_norm_fwd(x, w, b=None, eps: float = 1e-5, out=None, stream=None):
    """Layer norm over the last dimension (up to 16384): y = (x - mean) rstd w + b.  x [..., d] bfloat16 or
    float32; w, b fp32 [d] (b may be None).  Returns (y, mean, rstd), mean and rstd fp32 [...]."""
    code = _io_dtype(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    d, lead = x.shape[-1], x.shape[:-1]
    rows = x.numel() // d if d else 0
    _need(x, "x", x.dtype, x.shape, x.device)
    _need(w, "w", torch.float32, (d,), x.device)
    if b is not None:
        _need(b, "b", torch.float32, (d,), x.device)
    with _Call(x, stream) as call:
        if out is None:
            out = call.like(x)
        _need(out, "out", x.dtype, x.shape, x.device)
        mean = call.empty(lead, torch.float32)
        rstd = call.like(mean)
        st = lib.kda_layer_norm_fwd(_ptr(x), _ptr(w), _ptr(b), rows, d, float(eps), _ptr(out), _ptr(mean), _ptr(rstd),
                                    code, call.handle)
    _check(st, "kda_layer_norm_fwd")
    return out, mean, rstd


def kda_layer_norm_bwd(x, w, mean, rstd, dy, has_bias: bool = True, workspace=None, stream=None):
    """Gradients of kda_layer_norm_fwd; mean and rstd are the ones it returned, dy of x's dtype.  Returns a
    dict: dx of x's dtype, dw and (with has_bias, else None) dbias fp32 [d]."""
    code = _io_dtype(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    d, lead = x.shape[-1], x.shape[:-1]
    rows = x.numel() // d if d else 0
    _need(x, "x", x.dtype, x.shape, x.device)
    _need(dy, "dy", x.dtype, x.shape, x.device)
    _need(w, "w", torch.float32, (d,), x.device)
    _need(mean, "mean", torch.float32, lead, x.device)
    _need(rstd, "rstd", torch.float32, lead, x.device)
    with _Call(x, stream) as call:
        g = dict(dx=call.like(x), dw=call.like(w), dbias=call.like(w) if has_bias else None)
        ws, ws_bytes = call.workspace(workspace, kda_layer_norm_bwd_workspace_size(rows, d))
        st = lib.kda_layer_norm_bwd(_ptr(x), _ptr(w), _ptr(mean), _ptr(rstd), _ptr(dy), rows, d, _ptr(g["dx"]),
                                    _ptr(g["dw"]), _ptr(g["dbias"]), code, _ptr(ws), ws_bytes, call.handle)
    _check(st, "kda_layer_norm_bwd")
    return g


def _grad(d, like):
    """An incoming gradient as the kernels take it: of its tensor's dtype, dense; zeros where there is none."""
    return torch.zeros_like(like) if d is None else d.to(like.dtype).contiguous()


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A_log, B, C, skip, z, dt_bias, initial_state, cu_seqlens):
        out, last = kda_selective_scan_fwd(u, dt, A_log, B, C, cu_seqlens, skip=skip, z=z, dt_bias=dt_bias,
                                           initial_state=initial_state)
        ctx.save_for_backward(u, dt, A_log, B, C, skip, z, dt_bias, initial_state, cu_seqlens)
        ctx.set_materialize_grads(False)
        return out, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dlast):
        u, dt, A_log, B, C, skip, z, dt_bias, initial_state, cu_seqlens = ctx.saved_tensors
        g = kda_selective_scan_bwd(u, dt, A_log, B, C, cu_seqlens, _grad(dout, u), skip=skip, z=z, dt_bias=dt_bias,
                                   initial_state=initial_state, dfinal_state=None if dlast is None else dlast.contiguous())
        return (g["du"], g["ddt"], g["dA_log"], g["dB"], g["dC"], g["dskip"], g["dz"], g["ddt_bias"],
                g["dinitial_state"], None)


def selective_scan(u, dt, A_log, B, C, cu_seqlens, skip=None, z=None, dt_bias=None, initial_state=None):
    """kda_selective_scan_fwd as a differentiable function of every tensor but cu_seqlens; its backward is
    kda_selective_scan_bwd.  Returns (out, final_state).

    A training step of this, short_conv and layer_norm may be captured into a CUDA graph.  As for any autograd
    function, drop the results of earlier eager passes over the same leaves first: while one lives, the leaves'
    gradients belong to its stream, and a capture does not allow work there."""
    return _SelectiveScan.apply(u, dt, A_log, B, C, skip, z, dt_bias, initial_state, cu_seqlens)


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, initial_state, cu_seqlens, silu, l2norm):
        y, last = kda_short_conv_fwd(x, w, cu_seqlens, bias=bias, initial_state=initial_state, silu=silu, l2norm=l2norm)
        ctx.save_for_backward(x, w, bias, initial_state, cu_seqlens)
        ctx.silu, ctx.l2norm = silu, l2norm
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dlast):
        x, w, bias, initial_state, cu_seqlens = ctx.saved_tensors
        g = kda_short_conv_bwd(x, w, cu_seqlens, _grad(dy, x), bias=bias, initial_state=initial_state,
                               dfinal_state=None if dlast is None else dlast.contiguous(), silu=ctx.silu, l2norm=ctx.l2norm)
        return g["dx"], g["dw"], g["dbias"], g["dinitial_state"], None, None, None


def short_conv(x, w, cu_seqlens, bias=None, initial_state=None, silu: bool = False, l2norm: bool = False):
    """kda_short_conv_fwd as a differentiable function of x, w, bias and initial_state; its backward is
    kda_short_conv_bwd.  Returns (y, final_state)."""
    return _ShortConv.apply(x, w, bias, initial_state, cu_seqlens, bool(silu), bool(l2norm))


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, eps):
        y, mean, rstd = kda_layer_norm_fwd(x, w, b, eps=eps)
        ctx.save_for_backward(x, w, mean, rstd)
        ctx.has_bias = b is not None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, mean, rstd = ctx.saved_tensors
        g = kda_layer_norm_bwd(x, w, mean, rstd, _grad(dy, x), has_bias=ctx.has_bias)
        return g["dx"], g["dw"], g["dbias"], None


def layer_norm(x, w, b=None, eps: float = 1e-5):
    """kda_layer_norm_fwd as a differentiable function of x, w and b; its backward is kda_layer_norm_bwd."""
    return _LayerNorm.apply(x, w, b, float(eps))


def kda_launch_count() -> int:
    """Kernels launched through libkda by this process so far."""
    return int(lib.kda_launch_count())


def kda_set_prefill_path(path: int) -> None:
    """Which prefill kernel kda_chunk_fwd runs for d_k = d_v = 128: 0 chosen from the shapes,
    1 the cluster kernel (chunk records in the workspace), 2 one CTA per (sequence, head)."""
    _check(lib.kda_set_prefill_path(int(path)), "kda_set_prefill_path")


def kda_prefill_path(num_units: int, d_k: int, d_v: int) -> int:
    """The kernel kda_chunk_fwd would run now for num_units units: 1 (cluster) or 2 (per unit)."""
    return int(lib.kda_prefill_path(int(num_units), int(d_k), int(d_v)))


def kda_inject_stall(enable: bool, wait_limit_ns: int = 0) -> None:
    """Failure injection for tests: while enabled, prefill launches withhold chunk 0 and every
    device-side wait gives up after wait_limit_ns (the next kda_sync_check raises a timeout)."""
    _check(lib.kda_inject_stall(1 if enable else 0, int(wait_limit_ns)), "kda_inject_stall")


def kda_sync_check(stream=None, device=None) -> None:
    """Synchronise the stream and raise KDAError if a kernel recorded a device-side error."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    _check(lib.kda_sync_check(_stream_handle(stream, dev)), "kda_sync_check")
