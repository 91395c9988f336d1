"""Thin ctypes binding of the KDA C ABI (include/kda.h).

The functions named like the C entry points (``kda_chunk_prefill``,
``kda_chunk_prefill_ex``, ``kda_chunk_prefill_noalloc``, ``kda_decode_step``,
``kda_prepare_inputs``, ``kda_output_norm``, ``kda_decode_multi``, ``kda_ckpt_count``,
``kda_latent_append``, ``kda_latent_gather``, ``kda_latent_decode``, ``kda_latent_prefill``, ``kda_verify_draft``,
``kda_device_status``, ``kda_status_string``, ``kda_chunk_size``) only marshal
arguments: torch
tensors become raw device pointers, the current torch stream becomes the
``stream`` argument, and a negative status raises ``KdaError``.  ``prefill``,
``decode_step``, ``latent_gather``, ``latent_decode``, ``latent_prefill`` and ``verify_draft``
additionally allocate the output tensors with torch (a call with ``stream=`` from that stream's memory).

There is no fallback: if ``libkda.so`` is missing or cannot be loaded the
first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libkda.so")
_lock = threading.Lock()
_lib = None

KDA_OK = 0
KDA_ERR_INVALID_ARG = -1
KDA_ERR_UNSUPPORTED = -2
KDA_ERR_CUDA = -3
KDA_ERR_TIMEOUT = -4
KDA_ERR_RANGE = -5
KDA_OUT_BF16 = 0
KDA_OUT_F32 = 1
KDA_NOALLOC_MAX_SEQ_HEADS = 32
KDA_MAX_SEGMENTS = 64
KDA_DECAY_CHANNEL = 0
KDA_DECAY_HEAD = 1
KDA_DECAY_NONE = 2
KDA_CACHE_BF16 = 0
KDA_CACHE_E4M3 = 1
KDA_LATENT_DIM = 512
KDA_LATENT_ROPE = 64
KDA_LATENT_MAX_PAGE = 1024
KDA_LATENT_MAX_ROWS = 512
KDA_LATENT_MAX_TOKENS = 2**31 - 4096
KDA_VERIFY_MAX_DRAFT = 64

_vp = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64
_f = ctypes.c_float


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {kda_status_string(status)} ({status})")


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libkda.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(f"KDA CUDA library not built: {_LIB_PATH} is missing "
                                   "(run kimi_delta_attention_06_gb300.build.build())")
            lib = ctypes.CDLL(_LIB_PATH)
            for name in ("kda_chunk_prefill", "kda_chunk_prefill_noalloc"):
                fn = getattr(lib, name)
                fn.restype = _i
                fn.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _i, _vp, _vp, _i, _vp]
            lib.kda_chunk_prefill_ex.restype = _i
            lib.kda_chunk_prefill_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _i,
                                                 _vp, _vp, _i, _i, _vp, _vp, _vp, ctypes.c_float, _vp]
            lib.kda_chunk_prefill_segmented.restype = _i
            lib.kda_chunk_prefill_segmented.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i,
                                                        _vp, _vp, _i, _i, _i, _i, _vp, ctypes.c_float, _vp]
            lib.kda_chunk_prefill_segmented_ex.restype = _i
            lib.kda_chunk_prefill_segmented_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                                                           _i, _vp, _vp, _i, _i, _vp, _i, _vp, ctypes.c_float, _vp]
            lib.kda_segment_plan.restype = _i
            lib.kda_segment_plan.argtypes = [_i, _i, _i, _i, _vp, _vp, _i]
            lib.kda_prefill_clusters_at_once.restype = _i
            lib.kda_prefill_clusters_at_once.argtypes = []
            lib.kda_decode_step.restype = _i
            lib.kda_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]
            lib.kda_decode_multi.restype = _i
            lib.kda_decode_multi.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _vp, _i,
                                             _i, _i, _i, _i, _i, _i, _vp]
            lib.kda_prepare_inputs.restype = _i
            lib.kda_prepare_inputs.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                               _vp, _vp, _vp, _vp, _vp, _vp]
            lib.kda_output_norm.restype = _i
            lib.kda_output_norm.argtypes = [_vp, _i, _vp, ctypes.c_float, _vp, _i, _i, _i, _vp]
            lib.kda_latent_row_bytes.restype = _i
            lib.kda_latent_row_bytes.argtypes = [_i]
            lib.kda_latent_append.restype = _i
            lib.kda_latent_append.argtypes = [_vp, _i64, _vp, _i64, _vp, _i, _i, _i, _vp, _i, _vp]
            lib.kda_latent_gather.restype = _i
            lib.kda_latent_gather.argtypes = [_vp, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _vp, _i64, _vp, _i64,
                                              _vp]
            lib.kda_latent_decode.restype = _i
            lib.kda_latent_decode.argtypes = [_vp, _vp, _i, _i, _i, _vp, _i, _vp, _i, _i, _i, _f, _vp, _vp, _vp]
            lib.kda_latent_prefill.restype = _i
            lib.kda_latent_prefill.argtypes = [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp,
                                               _i, _i, _i, _i, _i, _f, _vp, _vp, _vp]
            lib.kda_verify_draft.restype = _i
            lib.kda_verify_draft.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp]
            lib.kda_ckpt_count.restype = ctypes.c_int64
            lib.kda_ckpt_count.argtypes = [_vp, _i, _i]
            lib.kda_ckpt_count_ex.restype = ctypes.c_int64
            lib.kda_ckpt_count_ex.argtypes = [_vp, _vp, _i, _i]
            lib.kda_device_status.restype = _i
            lib.kda_device_status.argtypes = [_vp]
            lib.kda_status_string.restype = ctypes.c_char_p
            lib.kda_status_string.argtypes = [_i]
            lib.kda_chunk_size.restype = _i
            lib.kda_chunk_size.argtypes = []
            lib.kda_debug_expire_wait.restype = _i
            lib.kda_debug_expire_wait.argtypes = [ctypes.c_ulonglong, _vp]
            lib.kda_debug_verify_cluster.restype = _i
            lib.kda_debug_verify_cluster.argtypes = [_i, _i, _i, _i]
            _lib = lib
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    """Device address of a contiguous tensor (the argument types make a pointer of it)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("KDA tensors must be contiguous")
    return t.data_ptr()


# The current stream's handle without building a Stream object: a few microseconds a call, which
# is as long as a small kernel runs.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _side(stream):
    """The torch stream of a ``stream`` argument, None where it is the current one."""
    if stream is None:
        return None
    handle = _stream(stream)
    if handle == _stream(None):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _empty(shape, dev, dtype, side=None):
    """An output for a call on the current stream or on ``side``.  Memory that the current stream's allocator
    hands out again may still be in use by work pending there, which nothing orders before a call on another
    stream: such a call's outputs come from its own stream's memory, and are marked as used here too."""
    if side is None:
        return torch.empty(shape, device=dev, dtype=dtype)
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(side):
        t = torch.empty(shape, device=dev, dtype=dtype)
    t.record_stream(here)
    return t


def _to_device(host: torch.Tensor, dev, side=None):
    """A device copy of a host array that lives as long as this call's launches need it, on ``side`` too: the
    copy is complete on return (pageable memory), and its memory is not handed out again before ``side`` gets
    past the work it holds by then."""
    t = host.to(dev)
    if side is not None:
        t.record_stream(side)
    return t


def _check(rc: int, what: str):
    if rc != KDA_OK:
        raise KdaError(rc, what)


def _bits16(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.bfloat16:
        raise TypeError(f"expected a bfloat16 tensor, got {t.dtype}")
    return t


# --- the C entry points, one to one --------------------------------------------------

def kda_status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def kda_chunk_size() -> int:
    return int(load().kda_chunk_size())


def kda_ckpt_count(cu_seqlens_host: torch.Tensor, ckpt_stride: int) -> int:
    cu = cu_seqlens_host.to(device="cpu", dtype=torch.int32).contiguous()
    n = load().kda_ckpt_count(ctypes.c_void_p(cu.data_ptr()), cu.numel() - 1, int(ckpt_stride))
    if n < 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_ckpt_count")
    return int(n)


def kda_ckpt_count_ex(cu_seqlens_host: torch.Tensor, start_pos_host, ckpt_stride: int) -> int:
    cu = cu_seqlens_host.to(device="cpu", dtype=torch.int32).contiguous()
    sp = None if start_pos_host is None else start_pos_host.to(device="cpu", dtype=torch.int32).contiguous()
    n = load().kda_ckpt_count_ex(ctypes.c_void_p(cu.data_ptr()), None if sp is None else ctypes.c_void_p(sp.data_ptr()),
                                 cu.numel() - 1, int(ckpt_stride))
    if n < 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_ckpt_count_ex")
    return int(n)


def _call_prefill(name, q, k, v, log_alpha, beta, init_state, cu_seqlens, cu_seqlens_host, num_seqs,
                  total_tokens, H, Dk, Dv, out, out_dtype, final_state, ckpt_states, ckpt_stride, stream):
    cu_host = cu_seqlens_host.to(device="cpu", dtype=torch.int32).contiguous()
    rc = getattr(load(), name)(
        _ptr(_bits16(q)), _ptr(_bits16(k)), _ptr(_bits16(v)), _ptr(log_alpha), _ptr(_bits16(beta)),
        _ptr(init_state), _ptr(cu_seqlens), ctypes.c_void_p(cu_host.data_ptr()),
        int(num_seqs), int(total_tokens), int(H), int(Dk), int(Dv),
        _ptr(out), int(out_dtype), _ptr(final_state), _ptr(ckpt_states), int(ckpt_stride),
        _stream(stream))
    _check(rc, name)


def kda_chunk_prefill(q, k, v, log_alpha, beta, init_state, cu_seqlens, cu_seqlens_host,
                      num_seqs: int, total_tokens: int, H: int, Dk: int, Dv: int,
                      out, out_dtype: int, final_state, ckpt_states, ckpt_stride: int, stream=None):
    _call_prefill("kda_chunk_prefill", q, k, v, log_alpha, beta, init_state, cu_seqlens, cu_seqlens_host,
                  num_seqs, total_tokens, H, Dk, Dv, out, out_dtype, final_state, ckpt_states, ckpt_stride, stream)


def kda_chunk_prefill_ex(q, k, v, log_alpha, beta, init_state, cu_seqlens, cu_seqlens_host,
                         num_seqs: int, total_tokens: int, H: int, Dk: int, Dv: int,
                         out, out_dtype: int, final_state, ckpt_states, ckpt_stride: int, decay: int,
                         start_pos=None, start_pos_host=None, out_norm_gamma=None, out_norm_eps: float = 1e-6,
                         stream=None):
    sp_host = None if start_pos_host is None else start_pos_host.to(device="cpu", dtype=torch.int32).contiguous()
    cu_host = cu_seqlens_host.to(device="cpu", dtype=torch.int32).contiguous()
    rc = load().kda_chunk_prefill_ex(
        _ptr(_bits16(q)), _ptr(_bits16(k)), _ptr(_bits16(v)), _ptr(log_alpha), _ptr(_bits16(beta)),
        _ptr(init_state), _ptr(cu_seqlens), ctypes.c_void_p(cu_host.data_ptr()),
        int(num_seqs), int(total_tokens), int(H), int(Dk), int(Dv),
        _ptr(out), int(out_dtype), _ptr(final_state), _ptr(ckpt_states), int(ckpt_stride), int(decay),
        _ptr(start_pos), None if sp_host is None else ctypes.c_void_p(sp_host.data_ptr()),
        _ptr(out_norm_gamma), float(out_norm_eps), _stream(stream))
    _check(rc, "kda_chunk_prefill_ex")


def kda_chunk_prefill_segmented(q, k, v, log_alpha, beta, init_state, total_tokens: int, H: int, Dk: int, Dv: int,
                                out, out_dtype: int, final_state, ckpt_states, ckpt_stride: int, decay: int,
                                start_pos: int, segments: int, out_norm_gamma=None, out_norm_eps: float = 1e-6,
                                stream=None):
    rc = load().kda_chunk_prefill_segmented(
        _ptr(_bits16(q)), _ptr(_bits16(k)), _ptr(_bits16(v)), _ptr(log_alpha), _ptr(_bits16(beta)),
        _ptr(init_state), int(total_tokens), int(H), int(Dk), int(Dv),
        _ptr(out), int(out_dtype), _ptr(final_state), _ptr(ckpt_states), int(ckpt_stride), int(decay),
        int(start_pos), int(segments), _ptr(out_norm_gamma), float(out_norm_eps), _stream(stream))
    _check(rc, "kda_chunk_prefill_segmented")


def kda_chunk_prefill_segmented_ex(q, k, v, log_alpha, beta, init_state, cu_seqlens_host, num_seqs: int,
                                   total_tokens: int, H: int, Dk: int, Dv: int, out, out_dtype: int, final_state,
                                   ckpt_states, ckpt_stride: int, decay: int, start_pos_host, segments: int,
                                   out_norm_gamma=None, out_norm_eps: float = 1e-6, stream=None):
    cu_host = cu_seqlens_host.to(device="cpu", dtype=torch.int32).contiguous()
    sp_host = None if start_pos_host is None else \
        torch.as_tensor(start_pos_host).to(device="cpu", dtype=torch.int32).contiguous()
    rc = load().kda_chunk_prefill_segmented_ex(
        _ptr(_bits16(q)), _ptr(_bits16(k)), _ptr(_bits16(v)), _ptr(log_alpha), _ptr(_bits16(beta)),
        _ptr(init_state), ctypes.c_void_p(cu_host.data_ptr()), int(num_seqs), int(total_tokens), int(H), int(Dk),
        int(Dv), _ptr(out), int(out_dtype), _ptr(final_state), _ptr(ckpt_states), int(ckpt_stride), int(decay),
        None if sp_host is None else ctypes.c_void_p(sp_host.data_ptr()), int(segments), _ptr(out_norm_gamma),
        float(out_norm_eps), _stream(stream))
    _check(rc, "kda_chunk_prefill_segmented_ex")


def kda_segment_plan(total_tokens: int, start_pos: int, segments: int, ckpt_stride: int = 0):
    """(bounds, ckpt_slots) of kda_chunk_prefill_segmented's plan: the segment bounds in tokens
    from the prompt's start, and for each of the prompt's checkpoints the slot it comes from,
    counted over run A's slots then run F's (empty when there are no checkpoints or one plain
    prefill runs)."""
    bounds = (ctypes.c_int32 * (KDA_MAX_SEGMENTS + 1))()
    cap = 1 << 16
    slots = (ctypes.c_int32 * cap)()
    P = load().kda_segment_plan(int(total_tokens), int(start_pos), int(segments), int(ckpt_stride),
                                ctypes.cast(bounds, ctypes.c_void_p), ctypes.cast(slots, ctypes.c_void_p), cap)
    _check(min(P, 0), "kda_segment_plan")
    n = kda_ckpt_count_ex(torch.tensor([0, int(total_tokens)], dtype=torch.int32),
                          torch.tensor([int(start_pos)], dtype=torch.int32), ckpt_stride) \
        if ckpt_stride > 0 and P >= 3 else 0
    return [int(x) for x in bounds[:P + 1]], [int(x) for x in slots[:n]]


def kda_prefill_clusters_at_once() -> int:
    n = load().kda_prefill_clusters_at_once()
    _check(min(n, 0), "kda_prefill_clusters_at_once")
    return int(n)


def segments_for(H: int, clusters_at_once: Optional[int] = None, num_seqs: int = 1) -> int:
    """Segments for kda_chunk_prefill_segmented(_ex): clusters_at_once // H + 1, at most 32, so
    that each run (P - 1 segments of a single sequence per head) fills the device in one wave.
    0 (a plain prefill) when that is below 3, or when the call's (sequence, head) pairs
    already fill the device (num_seqs * H >= clusters_at_once): splitting then only adds work.
    Beyond 32 segments the serial chain of segment states and the per-segment fixed costs
    grow while the runs shrink, and short segments are less likely to let their transitions
    be dropped."""
    n = kda_prefill_clusters_at_once() if clusters_at_once is None else int(clusters_at_once)
    H, num_seqs = max(1, int(H)), max(1, int(num_seqs))
    if num_seqs * H >= n:
        return 0
    p = min(n // H + 1, 32)
    return p if p >= 3 else 0


def kda_chunk_prefill_noalloc(q, k, v, log_alpha, beta, init_state, cu_seqlens, cu_seqlens_host,
                              num_seqs: int, total_tokens: int, H: int, Dk: int, Dv: int,
                              out, out_dtype: int, final_state, ckpt_states, ckpt_stride: int, stream=None):
    _call_prefill("kda_chunk_prefill_noalloc", q, k, v, log_alpha, beta, init_state, cu_seqlens,
                  cu_seqlens_host, num_seqs, total_tokens, H, Dk, Dv, out, out_dtype, final_state, ckpt_states,
                  ckpt_stride, stream)


def kda_decode_step(q, k, v, log_alpha, beta, state, out, out_dtype: int,
                    N: int, H: int, Dk: int, Dv: int, stream=None):
    rc = load().kda_decode_step(_ptr(_bits16(q)), _ptr(_bits16(k)), _ptr(_bits16(v)), _ptr(log_alpha),
                                _ptr(_bits16(beta)), _ptr(state), _ptr(out), int(out_dtype),
                                int(N), int(H), int(Dk), int(Dv), _stream(stream))
    _check(rc, "kda_decode_step")


def kda_decode_multi(q, k, v, log_alpha, beta, state_pool, num_slots: int, state_slots, num_tokens,
                     commit: int, out, out_dtype: int, N: int, K: int, H: int, Dk: int, Dv: int,
                     decay: int = KDA_DECAY_CHANNEL, stream=None):
    rc = load().kda_decode_multi(_ptr(_bits16(q)), _ptr(_bits16(k)), _ptr(_bits16(v)), _ptr(log_alpha),
                                 _ptr(_bits16(beta)), _ptr(state_pool), int(num_slots), _ptr(state_slots),
                                 _ptr(num_tokens), int(commit), _ptr(out), int(out_dtype),
                                 int(N), int(K), int(H), int(Dk), int(Dv), int(decay), _stream(stream))
    _check(rc, "kda_decode_multi")


def kda_prepare_inputs(xq, xk, xv, conv_w, conv_state, a_raw, b_raw, cu_seqlens, cu_seqlens_host,
                       num_seqs: int, total_tokens: int, H: int, D: int, conv_act: int,
                       q, k, v, log_alpha, beta, stream=None):
    cu_host = cu_seqlens_host.to(device="cpu", dtype=torch.int32).contiguous()
    rc = load().kda_prepare_inputs(_ptr(_bits16(xq)), _ptr(_bits16(xk)), _ptr(_bits16(xv)), _ptr(conv_w),
                                   _ptr(None if conv_state is None else _bits16(conv_state)), _ptr(a_raw),
                                   _ptr(_bits16(b_raw)), _ptr(cu_seqlens), ctypes.c_void_p(cu_host.data_ptr()),
                                   int(num_seqs), int(total_tokens), int(H), int(D), int(conv_act),
                                   _ptr(_bits16(q)), _ptr(_bits16(k)), _ptr(_bits16(v)), _ptr(log_alpha),
                                   _ptr(_bits16(beta)), _stream(stream))
    _check(rc, "kda_prepare_inputs")


def kda_output_norm(o, o_dtype: int, gamma, eps: float, y, total_tokens: int, H: int, Dv: int, stream=None):
    rc = load().kda_output_norm(_ptr(o), int(o_dtype), _ptr(gamma), float(eps), _ptr(_bits16(y)),
                                int(total_tokens), int(H), int(Dv), _stream(stream))
    _check(rc, "kda_output_norm")


# The calls below are as short as a small kernel, so each tensor is looked at once: its address (and
# its strides) come out of the function that checks its type, shape and layout.  The library sees
# addresses only, so a tensor that is smaller than the sizes of the call is refused here.
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def _dense(t: Optional[torch.Tensor], dtype, need: int, what: str):
    """Address of a contiguous tensor of at least `need` elements (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected a {dtype} tensor, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: KDA tensors must be contiguous")
    if t.numel() < need:
        raise ValueError(f"{what}: {need} elements are needed, {tuple(t.shape)} has {t.numel()}")
    return t.data_ptr()


def _rows2(t: torch.Tensor, dtype, rows: int, width: int, what: str):
    """(address, row stride in elements) of a 2-D tensor [rows or more, width or more] whose rows are contiguous;
    one row has any stride: `width`, which the checks pass."""
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected a {dtype} tensor, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] < rows or shape[1] < width:
        raise ValueError(f"{what}: expected a tensor [{rows}, {width}], got {tuple(shape)}")
    st = t.stride()
    if st[1] != 1 and t.numel():
        raise ValueError(f"{what}: the last dimension of a KDA tensor must be contiguous")
    return t.data_ptr(), st[0] if shape[0] > 1 else width


def _rows3(t: torch.Tensor, dtype, n0: int, n1: int, width: int, least0: int, what: str):
    """The same of a 3-D tensor [n0, n1, width] or more: (address, strides of its first two dimensions; of a
    single entry: least0 and width)."""
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected a {dtype} tensor, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[0] < n0 or shape[1] < n1 or shape[2] < width:
        raise ValueError(f"{what}: expected a tensor [{n0}, {n1}, {width}], got {tuple(shape)}")
    st = t.stride()
    if st[2] != 1 and t.numel():
        raise ValueError(f"{what}: the last dimension of a KDA tensor must be contiguous")
    return t.data_ptr(), st[0] if shape[0] > 1 else least0, st[1] if shape[1] > 1 else width


def _short(what: str, t: torch.Tensor, need: str):
    raise ValueError(f"{what}: expected a tensor {need}, got {tuple(t.shape)}")


def _on_gpu(*tensors):
    """After the other checks: the kernels follow these addresses."""
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("KDA tensors must be on the GPU")


def _out(t, dtype, need: int, what: str):
    """Address of an output that the caller brings."""
    p = _dense(t, dtype, need, what)
    _on_gpu(t)
    return p


def _host32(t):
    if isinstance(t, torch.Tensor) and t.dtype == torch.int32 and not t.is_cuda and t.is_contiguous():
        return t
    return torch.as_tensor(t).to(device="cpu", dtype=torch.int32).contiguous()


def _last32(t: torch.Tensor) -> int:
    """Last entry of a contiguous host int32 tensor (0 of an empty one), without an indexing call."""
    n = t.numel()
    return ctypes.c_int32.from_address(t.data_ptr() + 4 * (n - 1)).value if n else 0


def _host_offsets(t, seqs: int, what: str) -> torch.Tensor:
    t = _host32(t)
    if t.numel() < seqs + 1:
        raise ValueError(f"{what}: {seqs + 1} offsets are needed, got {t.numel()}")
    return t


_ROW_BYTES = {KDA_CACHE_BF16: 2 * (KDA_LATENT_DIM + KDA_LATENT_ROPE), KDA_CACHE_E4M3: KDA_LATENT_DIM + 2 * KDA_LATENT_ROPE + 16}


def kda_latent_row_bytes(cache_dtype: int) -> int:
    n = load().kda_latent_row_bytes(int(cache_dtype))
    _check(min(n, 0), "kda_latent_row_bytes")
    return int(n)


def _pages(cache: torch.Tensor, cache_dtype: int):
    """(pointer, num_pages, page_size) of a cache [num_pages, page_size, row bytes] uint8."""
    shape = cache.shape
    if cache.dtype != torch.uint8 or len(shape) != 3 or shape[2] != _ROW_BYTES.get(cache_dtype):
        raise ValueError("a latent cache is a uint8 tensor [num_pages, page_size, row bytes of its cache_dtype]")
    return _ptr(cache), shape[0], shape[1]


def kda_latent_append(c, k_rope, cache, cache_dtype: int, slots, total_tokens: int, stream=None):
    cp, ldc = _rows2(c, _BF16, total_tokens, KDA_LATENT_DIM, "c")
    rp, ldr = _rows2(k_rope, _BF16, total_tokens, KDA_LATENT_ROPE, "k_rope")
    p, num_pages, page_size = _pages(cache, cache_dtype)
    sp = _dense(slots, _I32, total_tokens, "slots")
    _on_gpu(c, k_rope, cache, slots)
    rc = load().kda_latent_append(cp, ldc, rp, ldr, p, cache_dtype, num_pages, page_size, sp, total_tokens, _stream(stream))
    if rc:
        _check(rc, "kda_latent_append")


# (the calls with the caller's outputs or, where `make` is set, with outputs of their own)

def _latent_gather(cache, cache_dtype, block_table, start_pos, cu_seqlens, cu_host, num_seqs, total_tokens, c, k_rope, stream,
                   make=False):
    if not make:
        cp, ldc = _rows2(c, _BF16, total_tokens, KDA_LATENT_DIM, "c")
        rp, ldr = _rows2(k_rope, _BF16, total_tokens, KDA_LATENT_ROPE, "k_rope")
    p, num_pages, page_size = _pages(cache, cache_dtype)
    tp, table = _dense(block_table, _I32, 0, "block_table"), block_table.shape
    if len(table) != 2 or table[0] < num_seqs:
        _short("block_table", block_table, f"[{num_seqs}, max_pages]")
    sp, cu = _dense(start_pos, _I32, num_seqs, "start_pos"), _dense(cu_seqlens, _I32, num_seqs + 1, "cu_seqlens")
    _on_gpu(cache, block_table, start_pos, cu_seqlens, c, k_rope)
    if make:
        dev, side = cache.device, _side(stream)
        if cu is None:
            cu_seqlens = _to_device(cu_host, dev, side)
            cu = cu_seqlens.data_ptr()
        c = _empty((total_tokens, KDA_LATENT_DIM), dev, _BF16, side)
        k_rope = _empty((total_tokens, KDA_LATENT_ROPE), dev, _BF16, side)
        cp, ldc, rp, ldr = c.data_ptr(), KDA_LATENT_DIM, k_rope.data_ptr(), KDA_LATENT_ROPE
    rc = load().kda_latent_gather(p, cache_dtype, num_pages, page_size, tp, table[1], sp, cu, cu_host.data_ptr(), num_seqs,
                                  total_tokens, cp, ldc, rp, ldr, _stream(stream))
    if rc:
        _check(rc, "kda_latent_gather")
    return c, k_rope


def _latent_decode(q, cache, cache_dtype, block_table, seq_lens, N, K, H, sm_scale, out, lse, stream, make=False, want_lse=False):
    qp = _dense(q, _BF16, N * K * H * 576, "q")
    if q.size(-1) != 576:
        _short("q", q, "[N, K, H, 576] (the absorbed query, then its position part)")
    p, num_pages, page_size = _pages(cache, cache_dtype)
    tp, table = _dense(block_table, _I32, 0, "block_table"), block_table.shape
    if len(table) != 2 or table[0] < N:
        _short("block_table", block_table, f"[{N}, max_pages]")
    sp = _dense(seq_lens, _I32, N, "seq_lens")
    _on_gpu(q, cache, block_table, seq_lens)
    if make:
        dev, side = q.device, _side(stream)
        out = _empty((N, K, H, KDA_LATENT_DIM), dev, _BF16, side)
        lse = _empty((N, K, H), dev, _F32, side) if want_lse else None
        op, lp = out.data_ptr(), lse.data_ptr() if want_lse else None
    else:
        op, lp = _out(out, _BF16, N * K * H * KDA_LATENT_DIM, "out"), _out(lse, _F32, N * K * H, "lse")
    rc = load().kda_latent_decode(qp, p, cache_dtype, num_pages, page_size, tp, table[1], sp, N, K, H, sm_scale, op, lp,
                                  _stream(stream))
    if rc:
        _check(rc, "kda_latent_decode")
    return out, lse


def _latent_prefill(q, k, v, k_rope, cu_q, cq, cu_k, ck, num_seqs, total_q, total_k, H, causal, sm_scale, out, lse, stream,
                    make=False, want_lse=False):
    qp = _dense(q, _BF16, total_q * H * 192, "q")
    if q.size(-1) != 192:
        _short("q", q, "[Tq, H, 192]")
    kp, ldk, hdk = _rows3(k, _BF16, total_k, H, 128, 128, "k")
    vp, ldv, hdv = _rows3(v, _BF16, total_k, H, 128, 128, "v")
    rp, ldr = _rows2(k_rope, _BF16, total_k, KDA_LATENT_ROPE, "k_rope")
    cqd, ckd = _dense(cu_q, _I32, num_seqs + 1, "cu_q"), _dense(cu_k, _I32, num_seqs + 1, "cu_k")
    _on_gpu(q, k, v, k_rope, cu_q, cu_k)
    if make:
        dev, side = q.device, _side(stream)
        if cqd is None:
            cu_q = _to_device(cq, dev, side)
            cqd = cu_q.data_ptr()
        if ckd is None:
            cu_k = _to_device(ck, dev, side)
            ckd = cu_k.data_ptr()
        out = _empty((total_q, H, 128), dev, _BF16, side)
        lse = _empty((total_q, H), dev, _F32, side) if want_lse else None
        op, lp = out.data_ptr(), lse.data_ptr() if want_lse else None
    else:
        op, lp = _out(out, _BF16, total_q * H * 128, "out"), _out(lse, _F32, total_q * H, "lse")
    rc = load().kda_latent_prefill(qp, kp, ldk, hdk, vp, ldv, hdv, rp, ldr, cqd, cq.data_ptr(), ckd, ck.data_ptr(), num_seqs,
                                   total_q, total_k, H, causal, sm_scale, op, lp, _stream(stream))
    if rc:
        _check(rc, "kda_latent_prefill")
    return out, lse


def _prob_rows(t, N: int, per: int, V: int, what: str):
    """(address, stride) of probabilities [N, per, V] whose N * per rows are one constant stride apart."""
    p, seq, ld = _rows3(t, _F32, N, per, V, -1, what)
    if per <= 1:
        return p, V if seq < 0 else seq
    if seq >= 0 and seq != per * ld:
        raise ValueError(f"{what}: the probability rows of consecutive sequences must be evenly spaced")
    return p, ld


def _verify_draft(target_probs, draft_probs, draft_tokens, num_draft, u_accept, u_sample, N, K, V, tokens, num_tokens,
                  stream, make=False):
    tp, ldp = _prob_rows(target_probs, N, K + 1, V, "target_probs")
    dp, ldq = (None, 0) if draft_probs is None else _prob_rows(draft_probs, N, K, V, "draft_probs")
    xp, up = _dense(draft_tokens, _I32, N * K, "draft_tokens"), _dense(u_accept, _F32, N * K, "u_accept")
    np_, sp = _dense(num_draft, _I32, N, "num_draft"), _dense(u_sample, _F32, N, "u_sample")
    _on_gpu(target_probs, draft_probs, draft_tokens, num_draft, u_accept, u_sample)
    if make:
        dev, side = target_probs.device, _side(stream)
        tokens, num_tokens = _empty((N, K + 1), dev, _I32, side), _empty((N,), dev, _I32, side)
        op, mp = tokens.data_ptr(), num_tokens.data_ptr()
    else:
        op, mp = _out(tokens, _I32, N * (K + 1), "tokens"), _out(num_tokens, _I32, N, "num_tokens")
    rc = load().kda_verify_draft(tp, ldp, dp, ldq, xp, np_, up, sp, N, K, V, op, mp, _stream(stream))
    if rc:
        _check(rc, "kda_verify_draft")
    return tokens, num_tokens


def kda_latent_gather(cache, cache_dtype: int, block_table, start_pos, cu_seqlens, cu_seqlens_host, num_seqs: int,
                      total_tokens: int, c, k_rope, stream=None):
    _latent_gather(cache, cache_dtype, block_table, start_pos, cu_seqlens,
                   _host_offsets(cu_seqlens_host, num_seqs, "cu_seqlens_host"), num_seqs, total_tokens, c, k_rope, stream)


def kda_latent_decode(q, cache, cache_dtype: int, block_table, seq_lens, N: int, K: int, H: int, sm_scale: float, out,
                      lse, stream=None):
    _latent_decode(q, cache, cache_dtype, block_table, seq_lens, N, K, H, sm_scale, out, lse, stream)


def kda_latent_prefill(q, k, v, k_rope, cu_q, cu_q_host, cu_k, cu_k_host, num_seqs: int, total_q: int, total_k: int,
                       H: int, causal: int, sm_scale: float, out, lse, stream=None):
    _latent_prefill(q, k, v, k_rope, cu_q, _host_offsets(cu_q_host, num_seqs, "cu_q_host"), cu_k,
                    _host_offsets(cu_k_host, num_seqs, "cu_k_host"), num_seqs, total_q, total_k, H, causal, sm_scale, out, lse,
                    stream)


def kda_verify_draft(target_probs, draft_probs, draft_tokens, num_draft, u_accept, u_sample, N: int, K: int, V: int,
                     tokens, num_tokens, stream=None):
    _verify_draft(target_probs, draft_probs, draft_tokens, num_draft, u_accept, u_sample, N, K, V, tokens, num_tokens,
                  stream)


def kda_debug_expire_wait(limit_ns: int, stream=None):
    _check(load().kda_debug_expire_wait(int(limit_ns), _stream(stream)), "kda_debug_expire_wait")


def kda_debug_verify_cluster(N: int, V: int, sms: int, clusters16: int) -> int:
    return int(load().kda_debug_verify_cluster(int(N), int(V), int(sms), int(clusters16)))


def kda_device_status(stream=None) -> int:
    return int(load().kda_device_status(_stream(stream)))


# --- conveniences: allocate outputs, then call the entry point ----------------------------

def prefill(q, k, v, log_alpha, beta, cu_seqlens_host, init_state=None, ckpt_stride: int = 0,
            out_dtype=torch.bfloat16, want_final: bool = True, cu_seqlens=None, stream=None,
            decay: int = KDA_DECAY_CHANNEL, start_pos_host=None, norm_gamma=None, norm_eps: float = 1e-6,
            segments: int = 0):
    """Allocate outputs and run kda_chunk_prefill (kda_chunk_prefill_ex for another decay
    layout, for start positions or with the output norm fused in: norm_gamma [H, Dv];
    kda_chunk_prefill_segmented(_ex) when segments > 0).
    Returns (out, final_state, ckpt_states)."""
    T, H, Dk = q.shape
    Dv = v.shape[2]
    cu_host = cu_seqlens_host.to(device="cpu", dtype=torch.int32).contiguous()
    N = cu_host.numel() - 1
    dev, side = q.device, _side(stream)
    if cu_seqlens is None:
        cu_seqlens = _to_device(cu_host, dev, side)
    out = _empty((T, H, Dv), dev, out_dtype, side)
    fin = _empty((N, H, Dk, Dv), dev, torch.float32, side) if want_final else None
    nck = kda_ckpt_count_ex(cu_host, start_pos_host, ckpt_stride) if ckpt_stride > 0 else 0
    ck = _empty((nck, H, Dk, Dv), dev, torch.float32, side) if ckpt_stride > 0 else None
    odt = KDA_OUT_F32 if out_dtype == torch.float32 else KDA_OUT_BF16
    if segments > 0 and N == 1:
        sp0 = 0 if start_pos_host is None else int(torch.as_tensor(start_pos_host).reshape(-1)[0])
        kda_chunk_prefill_segmented(q, k, v, log_alpha, beta, init_state, T, H, Dk, Dv, out, odt, fin,
                                    ck if nck > 0 else None, ckpt_stride, decay, sp0, segments, norm_gamma,
                                    norm_eps, stream)
    elif segments > 0:
        kda_chunk_prefill_segmented_ex(q, k, v, log_alpha, beta, init_state, cu_host, N, T, H, Dk, Dv, out, odt,
                                       fin, ck if nck > 0 else None, ckpt_stride, decay, start_pos_host, segments,
                                       norm_gamma, norm_eps, stream)
    elif decay == KDA_DECAY_CHANNEL and start_pos_host is None and norm_gamma is None:
        kda_chunk_prefill(q, k, v, log_alpha, beta, init_state, cu_seqlens, cu_host, N, T, H, Dk, Dv,
                          out, odt, fin, ck if nck > 0 else None, ckpt_stride, stream)
    else:
        sp = None if start_pos_host is None else start_pos_host.to(device="cpu", dtype=torch.int32).contiguous()
        kda_chunk_prefill_ex(q, k, v, log_alpha, beta, init_state, cu_seqlens, cu_host, N, T, H, Dk, Dv,
                             out, odt, fin, ck if nck > 0 else None, ckpt_stride, decay,
                             None if sp is None else _to_device(sp, dev, side), sp, norm_gamma, norm_eps, stream)
    return out, fin, ck


def decode_step(q, k, v, log_alpha, beta, state, out_dtype=torch.bfloat16, stream=None):
    """Run kda_decode_step in place on ``state``; returns the output tensor."""
    N, H, Dk = q.shape
    Dv = v.shape[2]
    out = _empty((N, H, Dv), q.device, out_dtype, _side(stream))
    kda_decode_step(q, k, v, log_alpha, beta, state, out,
                    KDA_OUT_F32 if out_dtype == torch.float32 else KDA_OUT_BF16, N, H, Dk, Dv, stream)
    return out


def latent_cache(num_pages: int, page_size: int, cache_dtype: int = KDA_CACHE_BF16, device="cuda") -> torch.Tensor:
    """A zeroed latent cache [num_pages, page_size, row bytes]."""
    return torch.zeros(num_pages, page_size, kda_latent_row_bytes(cache_dtype), dtype=torch.uint8, device=device)


def latent_append(c, k_rope, cache, cache_dtype: int, slots, stream=None):
    """Write tokens c [T, 512] and k_rope [T, 64] into the cache rows ``slots`` [T] (in place)."""
    kda_latent_append(c, k_rope, cache, cache_dtype, slots, c.shape[0], stream)


def latent_gather(cache, cache_dtype: int, block_table, cu_seqlens_host, cu_seqlens=None, start_pos=None, stream=None):
    """Read sequences back as dense rows; returns (c [T, 512], k_rope [T, 64]), bf16."""
    cu_host = _host32(cu_seqlens_host)
    return _latent_gather(cache, cache_dtype, block_table, start_pos, cu_seqlens, cu_host, cu_host.numel() - 1,
                          _last32(cu_host), None, None, stream, make=True)


def latent_decode(q, cache, cache_dtype: int, block_table, seq_lens, sm_scale: float, want_lse: bool = False, stream=None):
    """Absorbed latent attention of q [N, K, H, 576] over the cache; returns (out [N, K, H, 512] bf16,
    lse [N, K, H] fp32 or None)."""
    N, K, H, _ = q.shape
    return _latent_decode(q, cache, cache_dtype, block_table, seq_lens, N, K, H, sm_scale, None, None, stream, True, want_lse)


def latent_prefill(q, k, v, k_rope, cu_q_host, cu_k_host, sm_scale: float, causal: bool = True, cu_q=None, cu_k=None,
                   want_lse: bool = False, stream=None):
    """Expanded latent attention of q [Tq, H, 192] over k, v [Tk, H, 128] and k_rope [Tk, 64]; returns
    (out [Tq, H, 128] bf16, lse [Tq, H] fp32 or None)."""
    cq, ck = _host32(cu_q_host), _host32(cu_k_host)
    if ck.numel() != cq.numel():
        raise ValueError("cu_q_host and cu_k_host: offsets of one number of sequences")
    Tq, H, _ = q.shape
    return _latent_prefill(q, k, v, k_rope, cu_q, cq, cu_k, ck, cq.numel() - 1, Tq, k.shape[0], H, int(causal), sm_scale, None,
                           None, stream, True, want_lse)


def verify_draft(target_probs, draft_probs, draft_tokens, u_accept, u_sample, num_draft=None, stream=None):
    """Accept or reject draft_tokens [N, K] against target_probs [N, K + 1, V] (draft_probs [N, K, V] or None);
    returns (tokens [N, K + 1] int32, num_tokens [N] int32)."""
    N, K1, V = target_probs.shape
    if draft_tokens.size(-1) != K1 - 1 or u_accept.size(-1) != K1 - 1:
        _short("draft_tokens, u_accept", draft_tokens, f"[{N}, {K1 - 1}]")
    return _verify_draft(target_probs, draft_probs, draft_tokens, num_draft, u_accept, u_sample, N, K1 - 1, V, None, None, stream,
                         make=True)
