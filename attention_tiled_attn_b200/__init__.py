"""Fused attention forward for NVIDIA B200 (sm_100a): Python binding.

A thin ctypes layer over the C ABI declared in ``include/attn_b200.h``.  It only
marshals arguments (shapes, dtypes, data pointers, the current CUDA stream);
every step of the computation runs in the library's CUDA kernels.  There is
no CPU fallback: without the built library or a CUDA device the calls raise.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libattn_b200.so")

MODES = {"dot": 0, "rbf": 1, "sink": 2}
MASKS = {"none": 0, "causal": 1, "window": 2}
DTYPES = {torch.bfloat16: 0, torch.float32: 1}

ATTN_OK = 0


class AttnError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, status: int, text: str):
        super().__init__(f"attn status {status}: {text}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"CUDA library not built: {path} is missing (run python -m attention_tiled_attn_b200.build)")
    lib = ctypes.CDLL(path)
    vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, ci, vp, ci, ci, vp, ci, vp]
    lib.attn_fwd.restype = ci
    lib.attn_fwd_streaming.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, ci, vp, ci, ci, vp, ci, vp]
    lib.attn_fwd_streaming.restype = ci
    lib.attn_decode_indexed.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, ci, cf, vp, ci, ci, vp,
                                        vp]
    lib.attn_decode_indexed.restype = ci
    lib.attn_fwd_padded.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, ci, vp, ci, ci, vp, vp, vp, ci,
                                    vp]
    lib.attn_fwd_padded.restype = ci
    lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, ci, vp, ci, ci, ci,
                             vp, vp, vp, vp]
    lib.attn_bwd.restype = ci
    cz = ctypes.c_size_t
    lib.attn_kv4_write.argtypes = [vp] * 6 + [ci] * 6 + [cz] * 6 + [ci, vp, vp, ci, vp]
    lib.attn_kv4_write.restype = ci
    lib.attn_kv4_read.argtypes = [vp] * 6 + [ci] * 6 + [ci, vp, vp, ci, vp]
    lib.attn_kv4_read.restype = ci
    lib.attn_decode_kv4.argtypes = [vp] * 7 + [ci] * 8 + [cf, ci, vp, ci, ci, ci, vp, vp, cz, vp]
    lib.attn_decode_kv4.restype = ci
    lib.attn_decode_kv4_workspace_bytes.argtypes = []
    lib.attn_decode_kv4_workspace_bytes.restype = cz
    lib.attn_status_string.argtypes = [ci]
    lib.attn_status_string.restype = ctypes.c_char_p
    lib.attn_release_workspace.argtypes = []
    lib.attn_release_workspace.restype = None
    lib.attn_device_status.argtypes = [vp]
    lib.attn_device_status.restype = ci
    lib.attn_version.argtypes = []
    lib.attn_version.restype = ci
    lib.attn_exp2_poly_eval.argtypes = [vp, vp, ci, vp]
    lib.attn_exp2_poly_eval.restype = ci
    lib.attn_decode_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, ci, vp, ci, ci, vp, vp]
    lib.attn_decode_fwd_noalloc.restype = ci
    lib.attn_test_wait_timeout.argtypes = [ci, vp]
    lib.attn_test_wait_timeout.restype = ci
    lib.attn_test_fail_workspace_allocs.argtypes = [ci]
    lib.attn_test_fail_workspace_allocs.restype = ci
    lib.attn_decode_noalloc_scratch_bytes.argtypes = []
    lib.attn_decode_noalloc_scratch_bytes.restype = ctypes.c_size_t
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()


def _check(status: int):
    if status != ATTN_OK:
        raise AttnError(status, status_string(status))


def _check_kinds(mode: str, mask_kind: str, keep_first: int = 0, masks=None):
    """Rejects an unknown mode or mask kind, and kept keys without the streaming mask."""
    if mode not in MODES:
        raise ValueError(f"unknown mode {mode!r}")
    if mask_kind not in (masks or (*MASKS, "streaming")):
        raise ValueError(f"unknown mask kind {mask_kind!r}")
    if int(keep_first) != 0 and mask_kind != "streaming":
        raise ValueError("keep_first needs mask_kind 'streaming'")


def _same_device(ref: torch.Tensor, **tensors):
    """The library reads every pointer on ref's device; a tensor elsewhere is rejected."""
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} is on {t.device}, not on {ref.device} with q")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def attn_fwd_raw(q_ptr, k_ptr, v_ptr, out_ptr, lse_ptr, N, Hq, H, L, S, E, Ev, scale, mode, sink_ptr,
                 mask_kind, window, bias_ptr, dtype, stream_ptr) -> int:
    """The C entry point with integer pointers; returns the status code."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_fwd(c(q_ptr), c(k_ptr), c(v_ptr), c(out_ptr), c(lse_ptr), int(N), int(Hq), int(H), int(L),
                        int(S), int(E), int(Ev), float(scale), int(mode), c(sink_ptr), int(mask_kind),
                        int(window), c(bias_ptr), int(dtype), c(stream_ptr))


def attn_bwd_raw(q_ptr, k_ptr, v_ptr, out_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr, dv_ptr, dsink_ptr, N, Hq, H, L, S,
                 E, Ev, scale, mode, sink_ptr, mask_kind, window, stream_ptr, keep_first=0, bits_ptr=None,
                 start_ptr=None, end_ptr=None) -> int:
    """The backward C entry point with integer pointers; returns the status code."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_bwd(c(q_ptr), c(k_ptr), c(v_ptr), c(out_ptr), c(dout_ptr), c(lse_ptr), c(dq_ptr), c(dk_ptr),
                        c(dv_ptr), c(dsink_ptr), int(N), int(Hq), int(H), int(L), int(S), int(E), int(Ev),
                        float(scale), int(mode), c(sink_ptr), int(mask_kind), int(window), int(keep_first),
                        c(bits_ptr), c(start_ptr), c(end_ptr), c(stream_ptr))


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
             dout: torch.Tensor, *, scale: float, mode: str = "dot", sink: torch.Tensor | None = None,
             mask_kind: str = "none", window: int = 0, stream: torch.cuda.Stream | None = None, keep_first: int = 0,
             mask_bits: torch.Tensor | None = None, kv_start: torch.Tensor | None = None,
             kv_end: torch.Tensor | None = None):
    """Gradients (dq, dk, dv, dsink) of attn_fwd's output; float32 tensors, dsink None without a sink.

    q, k, v, out, dout: contiguous bfloat16 CUDA tensors (the forward's inputs and
    output, and the loss gradient of the output); lse: the forward's float32 lse.
    mask_kind "streaming" with window and keep_first, and mask_bits / kv_start /
    kv_end, mirror attn_fwd's arguments.
    """
    _check_kinds(mode, mask_kind, keep_first)
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous 4-D bfloat16 CUDA tensor")
    N, Hq, L, E = q.shape
    _, H, S, _ = k.shape
    Ev = v.shape[3]
    if tuple(out.shape) != (N, Hq, L, Ev) or tuple(dout.shape) != (N, Hq, L, Ev):
        raise ValueError("out and dout must be (N, Hq, L, Ev)")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (N, Hq, L) or not lse.is_cuda or not lse.is_contiguous():
        raise ValueError("lse must be the forward's float32 (N, Hq, L) tensor")
    if sink is not None and (sink.dtype != torch.float32 or sink.numel() != Hq or not sink.is_cuda
                             or not sink.is_contiguous()):
        raise ValueError("sink must be a contiguous CUDA float32 tensor of Hq values")
    for name, t, shape in (("mask_bits", mask_bits, (L, (S + 31) // 32)), ("kv_start", kv_start, (N,)),
                           ("kv_end", kv_end, (N,))):
        if t is not None and (not t.is_cuda or t.dtype != torch.int32 or tuple(t.shape) != shape
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of shape {shape}")
    _same_device(q, k=k, v=v, out=out, lse=lse, dout=dout, sink=sink, mask_bits=mask_bits, kv_start=kv_start,
                 kv_end=kv_end)
    dq = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    dk = torch.empty(k.shape, dtype=torch.float32, device=q.device)
    dv = torch.empty(v.shape, dtype=torch.float32, device=q.device)
    dsink = torch.empty(Hq, dtype=torch.float32, device=q.device) if sink is not None else None
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    if mask_kind == "streaming":
        kind, keep = MASKS["window"], int(keep_first)
    else:
        kind, keep = MASKS[mask_kind], 0
    with torch.cuda.device(q.device):
        st = load_library().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                                     _ptr(dv), _ptr(dsink), N, Hq, H, L, S, E, Ev, float(scale), MODES[mode],
                                     _ptr(sink), kind, int(window), keep, _ptr(mask_bits), _ptr(kv_start),
                                     _ptr(kv_end), ctypes.c_void_p(stream.cuda_stream))
    _check(st)
    return dq, dk, dv, dsink


def attn_fwd_padded_raw(q_ptr, k_ptr, v_ptr, out_ptr, lse_ptr, N, Hq, H, L, S, E, Ev, scale, mode, sink_ptr,
                        mask_kind, window, bits_ptr, start_ptr, end_ptr, dtype, stream_ptr) -> int:
    """The keep-bits / key-padding C entry point with integer pointers; returns the status code."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_fwd_padded(c(q_ptr), c(k_ptr), c(v_ptr), c(out_ptr), c(lse_ptr), int(N), int(Hq), int(H), int(L),
                               int(S), int(E), int(Ev), float(scale), int(mode), c(sink_ptr), int(mask_kind),
                               int(window), c(bits_ptr), c(start_ptr), c(end_ptr), int(dtype), c(stream_ptr))


def attn_fwd_streaming_raw(q_ptr, k_ptr, v_ptr, out_ptr, lse_ptr, N, Hq, H, L, S, E, Ev, scale, mode, sink_ptr,
                           window, keep_first, bias_ptr, dtype, stream_ptr) -> int:
    """The streaming-mask C entry point with integer pointers; returns the status code."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_fwd_streaming(c(q_ptr), c(k_ptr), c(v_ptr), c(out_ptr), c(lse_ptr), int(N), int(Hq), int(H),
                                  int(L), int(S), int(E), int(Ev), float(scale), int(mode), c(sink_ptr),
                                  int(window), int(keep_first), c(bias_ptr), int(dtype), c(stream_ptr))


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale: float, mode: str = "dot",
             sink: torch.Tensor | None = None, mask_kind: str = "none", window: int = 0,
             bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
             lse: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None, keep_first: int = 0,
             mask_bits: torch.Tensor | None = None, kv_start: torch.Tensor | None = None,
             kv_end: torch.Tensor | None = None):
    """out = softmax(z + B) V on the GPU.  Returns (out, lse).

    q (N, Hq, L, E), k (N, H, S, E), v (N, H, S, Ev): contiguous CUDA tensors,
    all bfloat16 or all float32.  sink: (Hq,) float32 or None.  bias: (L, S)
    float32 or None.  mode: "dot", "rbf" or "sink"; mask_kind: "none",
    "causal", "window" or "streaming" (the first ``keep_first`` keys plus the
    last ``window`` keys, through attn_fwd_streaming).  out/lse may be given
    (contiguous, right shape).  mask_bits (L, ceil(S/32)) int32 (bit j%32 of
    word j/32 set: row may attend key j), kv_start / kv_end (N,) int32 key
    padding: any of them routes the call through attn_fwd_padded (no bias).
    """
    _check_kinds(mode, mask_kind, keep_first)
    load_library()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D tensor")
    if q.dtype not in DTYPES or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share dtype bfloat16 or float32")
    N, Hq, L, E = q.shape
    Nk, H, S, Ek = k.shape
    Nv, Hv, Sv, Ev = v.shape
    if Nk != N or Nv != N or Hv != H or Sv != S or Ek != E:
        raise ValueError("inconsistent q/k/v shapes")
    if sink is not None and (sink.dtype != torch.float32 or sink.numel() != Hq or not sink.is_cuda
                             or not sink.is_contiguous()):
        raise ValueError("sink must be a contiguous CUDA float32 tensor of Hq values")
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (L, S) or not bias.is_cuda
                             or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous CUDA float32 (L, S) tensor")
    if out is None:
        out = torch.empty((N, Hq, L, Ev), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((N, Hq, L), dtype=torch.float32, device=q.device)
    if tuple(out.shape) != (N, Hq, L, Ev) or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out has the wrong shape/dtype")
    if tuple(lse.shape) != (N, Hq, L) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse has the wrong shape/dtype")
    _same_device(q, k=k, v=v, out=out, lse=lse, sink=sink, bias=bias, mask_bits=mask_bits, kv_start=kv_start,
                 kv_end=kv_end)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    with torch.cuda.device(q.device):
        lib = load_library()
        common = (_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), N, Hq, H, L, S, E, Ev, float(scale), MODES[mode],
                  _ptr(sink))
        tail = (_ptr(bias), DTYPES[q.dtype], ctypes.c_void_p(stream.cuda_stream))
        padded = mask_bits is not None or kv_start is not None or kv_end is not None
        if padded:
            if bias is not None or mask_kind == "streaming":
                raise ValueError("mask_bits / kv_start / kv_end combine with none, causal or window masks only, "
                                 "without a bias")
            for name, t, shape in (("mask_bits", mask_bits, (L, (S + 31) // 32)), ("kv_start", kv_start, (N,)),
                                   ("kv_end", kv_end, (N,))):
                if t is not None and (not t.is_cuda or t.dtype != torch.int32 or tuple(t.shape) != shape
                                      or not t.is_contiguous()):
                    raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of shape {shape}")
            st = lib.attn_fwd_padded(*common, MASKS[mask_kind], int(window), _ptr(mask_bits), _ptr(kv_start),
                                     _ptr(kv_end), *tail[1:])
        elif mask_kind == "streaming":
            st = lib.attn_fwd_streaming(*common, int(window), int(keep_first), *tail)
        else:
            st = lib.attn_fwd(*common, MASKS[mask_kind], int(window), *tail)
    _check(st)
    return out, lse


def attn_decode_indexed_raw(q_ptr, k_ptr, v_ptr, out_ptr, lse_ptr, idx_ptr, n_sel, N, Hq, H, L, S, E, Ev, scale,
                            sink_ptr, mask_kind, window, bias_ptr, stream_ptr) -> int:
    """The index-set decode entry point with integer pointers; returns the status code."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_decode_indexed(c(q_ptr), c(k_ptr), c(v_ptr), c(out_ptr), c(lse_ptr), c(idx_ptr), int(n_sel),
                                   int(N), int(Hq), int(H), int(L), int(S), int(E), int(Ev), float(scale),
                                   c(sink_ptr), int(mask_kind), int(window), c(bias_ptr), c(stream_ptr))


def attn_decode_indexed(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, key_idx: torch.Tensor, *, scale: float,
                        sink: torch.Tensor | None = None, mask_kind: str = "none", window: int = 0,
                        bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        lse: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Exact decode attention over listed keys.  Returns (out, lse).

    q (N, Hq, L, E), k (N, H, S, E), v (N, H, S, Ev): contiguous bfloat16 CUDA
    tensors with (Hq/H)*L <= 16.  key_idx (N, H, n_sel) int32 CUDA tensor of key
    positions; entries outside [0, S) select nothing.  sink, bias, mask_kind
    ("none", "causal", "window") and window as in attn_fwd.
    """
    _check_kinds("dot", mask_kind, masks=MASKS)
    for name, t in (("q", q), ("k", k), ("v", v), ("key_idx", key_idx)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4 or key_idx.dim() != 3:
        raise ValueError("q, k, v must be 4-D and key_idx 3-D")
    if q.dtype != torch.bfloat16 or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must be bfloat16")
    if key_idx.dtype != torch.int32:
        raise ValueError("key_idx must be int32")
    N, Hq, L, E = q.shape
    _, H, S, _ = k.shape
    Ev = v.shape[3]
    if tuple(key_idx.shape[:2]) != (N, H):
        raise ValueError("key_idx must be (N, H, n_sel)")
    if sink is not None and (sink.dtype != torch.float32 or sink.numel() != Hq or not sink.is_cuda
                             or not sink.is_contiguous()):
        raise ValueError("sink must be a contiguous CUDA float32 tensor of Hq values")
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (L, S) or not bias.is_cuda
                             or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous CUDA float32 (L, S) tensor")
    if out is None:
        out = torch.empty((N, Hq, L, Ev), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((N, Hq, L), dtype=torch.float32, device=q.device)
    if tuple(out.shape) != (N, Hq, L, Ev) or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out has the wrong shape/dtype")
    if tuple(lse.shape) != (N, Hq, L) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse has the wrong shape/dtype")
    _same_device(q, k=k, v=v, key_idx=key_idx, out=out, lse=lse, sink=sink, bias=bias)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    with torch.cuda.device(q.device):
        st = load_library().attn_decode_indexed(
            _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(key_idx), key_idx.shape[2], N, Hq, H, L, S, E, Ev,
            float(scale), _ptr(sink), MASKS[mask_kind], int(window), _ptr(bias), ctypes.c_void_p(stream.cuda_stream))
    _check(st)
    return out, lse


class KV4Cache(NamedTuple):
    """A key/value cache in 4 bits: uint8 CUDA tensors, contiguous, `capacity` rows of every (batch, KV head).

    k_codes (N, H, capacity, E/2), k_scales (N, H, capacity, E/16), v_codes
    (N, H, capacity, Ev/2), v_scales (N, H, capacity, Ev/16); the format is
    described in include/attn_b200.h.  A plain tuple of the four does as well.
    """

    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def kv4_cache(N: int, H: int, capacity: int, E: int, Ev: int | None = None, device="cuda") -> KV4Cache:
    """An empty 4-bit cache (all rows 0).  capacity is rounded up to a multiple of 16."""
    Ev = E if Ev is None else Ev
    C = -(-int(capacity) // 16) * 16
    return KV4Cache(*(torch.zeros((N, H, C, w), dtype=torch.uint8, device=device)
                      for w in (E // 2, E // 16, Ev // 2, Ev // 16)))


def _cache_shape(cache):
    """Checks a 4-bit cache's tensors and returns (N, H, capacity, E, Ev, device)."""
    kc, ks, vc, vs = cache
    N, H, C, half = kc.shape
    half_v = vc.shape[3]
    if ks.shape != (N, H, C, half // 8) or vc.shape != (N, H, C, half_v) or vs.shape != (N, H, C, half_v // 8):
        raise ValueError("the cache's tensors must be (N, H, C, E/2), (N, H, C, E/16), (N, H, C, Ev/2), (N, H, C, Ev/16)")
    dev = kc.device
    if not (kc.is_cuda and ks.device == dev and vc.device == dev and vs.device == dev
            and kc.dtype is ks.dtype is vc.dtype is vs.dtype is torch.uint8
            and kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
        raise ValueError("the cache must be contiguous uint8 CUDA tensors on one device")
    if max(N, H, C, 2 * half, 2 * half_v) >= 2**31:  # the C interface's sizes; see _int32
        raise ValueError("the cache's sizes must fit in 32 bits")
    return N, H, C, 2 * half, 2 * half_v, dev


def _check_index(name: str, t, N: int, device):
    if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != N or t.device != device
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape ({N},) on {device}")


def _int32(**values):
    """The C interface takes 32-bit sizes: a larger value is rejected, not cut."""
    for name, x in values.items():
        if not -2**31 <= x < 2**31:
            raise ValueError(f"{name} must fit in 32 bits")


def _address(t):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device) -> int:
    """The cudaStream_t of the device's current stream."""
    return torch.cuda.current_stream(device).cuda_stream if _raw_stream is None else _raw_stream(device.index)


def _elsewhere(device, stream) -> bool:
    """Whether a call has to change the current device or stream first."""
    return stream is not None or torch.cuda.current_device() != device.index


@contextlib.contextmanager
def _on(device, stream):
    """Makes `device` and `stream` (None: the device's current stream) the current ones, so that what a call
    allocates belongs to the stream that it is used on."""
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, not on {device} with the tensors")
    with torch.cuda.device(device) if stream is None else torch.cuda.stream(stream):
        yield


def attn_kv4_write_raw(k_ptr, v_ptr, kc_ptr, ks_ptr, vc_ptr, vs_ptr, N, H, L, C, E, Ev, k_strides, v_strides, start,
                       pos_ptr, count_ptr, dtype, stream_ptr) -> int:
    """The cache-writing C entry point with integer pointers; returns the status code."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_kv4_write(c(k_ptr), c(v_ptr), c(kc_ptr), c(ks_ptr), c(vc_ptr), c(vs_ptr), int(N), int(H), int(L),
                              int(C), int(E), int(Ev), *map(int, k_strides), *map(int, v_strides), int(start),
                              c(pos_ptr), c(count_ptr), int(dtype), c(stream_ptr))


def attn_kv4_read_raw(kc_ptr, ks_ptr, vc_ptr, vs_ptr, k_ptr, v_ptr, N, H, rows, C, E, Ev, start, pos_ptr, len_ptr,
                      dtype, stream_ptr) -> int:
    """The cache-reading C entry point with integer pointers; returns the status code."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_kv4_read(c(kc_ptr), c(ks_ptr), c(vc_ptr), c(vs_ptr), c(k_ptr), c(v_ptr), int(N), int(H), int(rows),
                             int(C), int(E), int(Ev), int(start), c(pos_ptr), c(len_ptr), int(dtype), c(stream_ptr))


def attn_decode_kv4_raw(q_ptr, kc_ptr, ks_ptr, vc_ptr, vs_ptr, out_ptr, lse_ptr, N, Hq, H, L, S, C, E, Ev, scale, mode,
                        sink_ptr, mask_kind, window, keep_first, len_ptr, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The 4-bit decode C entry point with integer pointers; returns the status code."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_decode_kv4(c(q_ptr), c(kc_ptr), c(ks_ptr), c(vc_ptr), c(vs_ptr), c(out_ptr), c(lse_ptr), int(N),
                               int(Hq), int(H), int(L), int(S), int(C), int(E), int(Ev), float(scale), int(mode),
                               c(sink_ptr), int(mask_kind), int(window), int(keep_first), c(len_ptr), c(ws_ptr),
                               int(ws_bytes), c(stream_ptr))


def attn_kv4_write(cache, k: torch.Tensor, v: torch.Tensor, *, start: int = 0, pos: torch.Tensor | None = None,
                   count: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> None:
    """Rounds new rows k (N, H, L, E), v (N, H, L, Ev) to 4 bits and stores them in the cache.

    k, v: bfloat16 or float32 CUDA tensors, the last dimension contiguous, any
    other strides that are multiples of 16 bytes (a slice of a fused projection,
    transposed, needs no copy).  Row l of sequence n goes to cache row pos[n] + l
    (pos (N,) int32 CUDA), or start + l without pos; with count (N,) int32 only
    its first count[n] rows are written.  Rows outside the cache are not written.
    """
    N, H, C, E, Ev, dev = _cache_shape(cache)
    ks, vs = k.shape, v.shape
    if len(ks) != 4 or ks[:2] != (N, H) or vs != (N, H, ks[2], Ev) or ks[3] != E:
        raise ValueError("k and v must be (N, H, L, E) and (N, H, L, Ev) with the cache's N, H, E and Ev")
    if k.dtype not in DTYPES or v.dtype is not k.dtype:
        raise ValueError("k, v must share dtype bfloat16 or float32")
    if k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be on {dev} with the cache")
    kst, vst = k.stride(), v.stride()
    if kst[3] != 1 or vst[3] != 1:
        raise ValueError("the last dimension of k and v must be contiguous")
    _check_index("pos", pos, N, dev)
    _check_index("count", count, N, dev)
    _int32(start=start, rows=ks[2])
    kc, ksc, vc, vsc = cache
    args = (k.data_ptr(), v.data_ptr(), kc.data_ptr(), ksc.data_ptr(), vc.data_ptr(), vsc.data_ptr(), N, H, ks[2], C, E, Ev,
            kst[0], kst[1], kst[2], vst[0], vst[1], vst[2], start, _address(pos), _address(count), DTYPES[k.dtype])
    lib = load_library()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            st = lib.attn_kv4_write(*args, _stream_handle(dev))
    else:
        st = lib.attn_kv4_write(*args, _stream_handle(dev))
    _check(st)


def attn_kv4_read(cache, rows: int, *, start: int = 0, pos: torch.Tensor | None = None,
                  kv_len: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
                  k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None):
    """`rows` cache rows of every (batch, KV head) from row pos[n] (or start): (k, v) of shapes
    (N, H, rows, E) and (N, H, rows, Ev) in `dtype` (bfloat16 or float32; both hold the values exactly).

    Rows at or after kv_len[n] ((N,) int32 CUDA) and rows outside the cache come
    back as 0.  k_out and v_out may be given (contiguous, of `dtype`).
    """
    N, H, C, E, Ev, dev = _cache_shape(cache)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_kv4_read(cache, rows, start=start, pos=pos, kv_len=kv_len, dtype=dtype, k_out=k_out, v_out=v_out)
    if dtype not in DTYPES:
        raise ValueError("dtype must be bfloat16 or float32")
    _int32(rows=rows, start=start)
    _check_index("pos", pos, N, dev)
    _check_index("kv_len", kv_len, N, dev)
    k_out = _output("k_out", k_out, (N, H, rows, E), dtype, dev)
    v_out = _output("v_out", v_out, (N, H, rows, Ev), dtype, dev)
    kc, ks, vc, vs = cache
    _check(load_library().attn_kv4_read(
        kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), N, H, rows, C, E, Ev,
        start, _address(pos), _address(kv_len), DTYPES[dtype], _stream_handle(dev)))
    return k_out, v_out


def _output(name, t, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")
    return t


KV4_WORKSPACE_ZERO = 4096  # leading bytes of a workspace that are zero before its first use
_kv4_workspaces: dict = {}  # (device index, stream handle) -> workspace


def kv4_workspace(device="cuda") -> torch.Tensor:
    """A workspace for attn_decode_kv4, ready for use on the current stream (its counters are zeroed there)."""
    ws = torch.empty(load_library().attn_decode_kv4_workspace_bytes(), dtype=torch.uint8, device=device)
    ws[:KV4_WORKSPACE_ZERO].zero_()
    return ws


def _kv4_stream_workspace(device, handle):
    """The workspace of calls on one stream.  A captured call gets one of its own, which lives in the graph's
    memory: replays may overlap calls on the stream that the graph was captured on."""
    if torch.cuda.is_current_stream_capturing():
        return kv4_workspace(device)
    key = (device.index, handle)
    ws = _kv4_workspaces.get(key)
    if ws is None:
        ws = _kv4_workspaces.setdefault(key, kv4_workspace(device))
    return ws


def attn_decode_kv4(q: torch.Tensor, cache, *, scale: float, length: int | None = None,
                    kv_len: torch.Tensor | None = None, mode: str = "dot", sink: torch.Tensor | None = None,
                    mask_kind: str = "none", window: int = 0, keep_first: int = 0, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None):
    """Decode attention straight from a 4-bit cache.  Returns (out, lse).

    q (N, Hq, L, E): contiguous bfloat16 CUDA tensor with (Hq/H)*L <= 16.  length:
    cached rows of the longest sequence (default: the capacity); kv_len (N,) int32:
    the rows of each sequence, at most length.  Query row i of sequence n is at
    position kv_len[n] - L + i, so the L new tokens' own rows are written first
    (attn_kv4_write) and counted.  mode, sink, mask_kind ("none", "causal",
    "window", "streaming"), window and keep_first as in attn_fwd.  workspace: a
    kv4_workspace() that no overlapping call uses (default: one per stream, and one
    of its own for a captured call).
    """
    _check_kinds(mode, mask_kind, keep_first)
    N, H, C, E, Ev, dev = _cache_shape(cache)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_decode_kv4(q, cache, scale=scale, length=length, kv_len=kv_len, mode=mode, sink=sink,
                                   mask_kind=mask_kind, window=window, keep_first=keep_first, out=out, lse=lse,
                                   workspace=workspace)
    if q.dim() != 4 or q.dtype is not torch.bfloat16 or q.device != dev or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous 4-D bfloat16 tensor on {dev} with the cache")
    Nq, Hq, L, Eq = q.shape
    if Nq != N or Eq != E:
        raise ValueError("q has another batch or head dimension than the cache")
    S = C if length is None else length
    _int32(length=S, window=window, keep_first=keep_first)
    _check_index("kv_len", kv_len, N, dev)
    if sink is not None and (sink.dtype is not torch.float32 or sink.numel() != Hq or sink.device != dev
                             or not sink.is_contiguous()):
        raise ValueError(f"sink must be a contiguous float32 tensor of Hq values on {dev}")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    out = torch.empty_like(q) if out is None and E == Ev else _output("out", out, (N, Hq, L, Ev), torch.bfloat16, dev)
    lse = _output("lse", lse, (N, Hq, L), torch.float32, dev)
    handle = _stream_handle(dev)
    ws = _kv4_stream_workspace(dev, handle) if workspace is None else workspace
    kc, ks, vc, vs = cache
    _check(load_library().attn_decode_kv4(
        q.data_ptr(), kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), out.data_ptr(), lse.data_ptr(), N, Hq,
        H, L, S, C, E, Ev, scale, MODES[mode], _address(sink), MASKS["window" if mask_kind == "streaming" else mask_kind],
        window, keep_first, _address(kv_len), ws.data_ptr(), ws.nbytes, handle))
    return out, lse


def attn_decode_fwd_noalloc_raw(q_ptr, k_ptr, v_ptr, out_ptr, lse_ptr, N, Hq, H, L, S, E, Ev, scale, mode,
                                sink_ptr, mask_kind, window, bias_ptr, stream_ptr) -> int:
    """The allocation-free decode entry point with integer pointers; returns the status.

    For callers that may not allocate device memory while running: the
    decode partials live in a fixed scratch array inside the library instead
    of an allocated workspace (see include/attn_b200.h)."""
    lib = load_library()
    c = lambda p: None if p is None else ctypes.c_void_p(int(p))  # noqa: E731
    return lib.attn_decode_fwd_noalloc(c(q_ptr), c(k_ptr), c(v_ptr), c(out_ptr), c(lse_ptr), int(N), int(Hq),
                                       int(H), int(L), int(S), int(E), int(Ev), float(scale), int(mode),
                                       c(sink_ptr), int(mask_kind), int(window), c(bias_ptr), c(stream_ptr))


def exp2_poly_eval(x: torch.Tensor) -> torch.Tensor:
    """The softmax's software 2^x applied on the GPU to a float32 CUDA tensor (verification)."""
    assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()
    y = torch.empty_like(x)
    _check(load_library().attn_exp2_poly_eval(_ptr(x), _ptr(y), x.numel(),
                                              ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    return y


def decode_noalloc_scratch_bytes() -> int:
    return int(load_library().attn_decode_noalloc_scratch_bytes())


def inject_wait_timeout(limit_cycles: int, stream: torch.cuda.Stream | None = None) -> int:
    """Failure-path check: a kernel whose one bounded wait runs out (returns the launch status)."""
    s = stream or torch.cuda.current_stream()
    return load_library().attn_test_wait_timeout(int(limit_cycles), ctypes.c_void_p(s.cuda_stream))


def inject_workspace_failures(count: int) -> int:
    """Failure-path check: the next `count` workspace allocations fail (returns the status)."""
    return load_library().attn_test_fail_workspace_allocs(int(count))


def device_status(stream: torch.cuda.Stream | None = None) -> int:
    """Synchronises the stream and returns (and clears) the kernels' fault status."""
    s = stream or torch.cuda.current_stream()
    return load_library().attn_device_status(ctypes.c_void_p(s.cuda_stream))


def release_workspace():
    load_library().attn_release_workspace()
    _kv4_workspaces.clear()


def version() -> int:
    return load_library().attn_version()
