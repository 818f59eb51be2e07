"""Exact IO-aware tiled attention for GB300 (sm_103a).

Python binding of the C ABI in include/fa.h.  Functions with the C names
(``fa_fwd``, ``fa_bwd``, ``fa_bwd_workspace_size``, ``fa_get_last_device_error``,
``fa_strerror``, ...) marshal torch tensors to pointers and call the library;
``forward`` / ``backward`` also allocate the outputs.  Every step of the
computation runs in the library's CUDA kernels: torch only provides device
memory and the current stream.

Layouts: dense tensors are [B, H, N, D]; packed variable-length batches are
[H, T, D] with int32 ``cu_seqlens`` [B + 1] on the device and ``max_seqlen``.
"""

import contextlib
import math
from typing import NamedTuple

import torch

from ._lib import FA_BF16, FA_F16, FA_F32, FAError, lib, library_path  # noqa: F401

__all__ = ["fa_fwd", "fa_bwd", "fa_bwd_workspace_size", "fa_get_last_device_error", "fa_strerror",
           "fa_set_wait_limit_ns", "fa_selftest_wait_timeout", "fa_selftest_tile", "fa_path_name", "fa_launch_count", "fa_bwd_static_ws", "fa_bwd_time_main_kernel", "forward", "backward",
           "fa_decode", "fa_decode_workspace_size", "decode", "fa_fwd_dropout", "fa_bwd_dropout",
           "fa_bwd_deterministic", "fa_probe_ex2_rate", "FAError",
           "Cache8", "cache_alloc", "fa_cache_write", "fa_cache_read", "cache_read", "fa_decode_cache",
           "fa_decode_cache_workspace_size", "decode_cache", "fa_decode_shared", "fa_decode_shared_workspace_size",
           "decode_shared"]

_DT = {torch.bfloat16: FA_BF16, torch.float32: FA_F32, torch.float16: FA_F16}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dims(q, cu_seqlens, max_seqlen):
    """(B, H, N, D, T) from the tensor shapes."""
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("dense tensors must be [B, H, N, D]")
        B, H, N, D = q.shape
        return B, H, N, D, 0
    if q.dim() != 3:
        raise ValueError("packed tensors must be [H, T, D]")
    if max_seqlen is None:
        raise ValueError("packed input needs max_seqlen")
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    H, T, D = q.shape
    return cu_seqlens.numel() - 1, H, int(max_seqlen), D, T


def _check(*tensors):
    ref = tensors[0]
    for t in tensors:
        if t is None:
            continue
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if t.device != ref.device:
            raise ValueError("tensors must be on one device")


def fa_strerror(status):
    return lib().fa_strerror(int(status)).decode()


def fa_path_name(dtype, D):
    r = lib().fa_path_name(_DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype), int(D))
    return None if r is None else r.decode()


def fa_launch_count():
    return int(lib().fa_launch_count())


def fa_bwd_time_main_kernel(start_event, stop_event):
    """Have the next fa_bwd on this thread record the two torch.cuda.Events
    (already recorded once, so they exist) around its main gradient kernel."""
    lib().fa_bwd_time_main_kernel(start_event.cuda_event, stop_event.cuda_event)


def fa_probe_ex2_rate(iters=4096, stream=None):
    """Measured ex2.approx throughput, exponentials per clock per SM (see
    fa_probe_ex2_rate in include/fa.h).  Synchronises the stream."""
    import ctypes
    out = ctypes.c_double(0.0)
    st = lib().fa_probe_ex2_rate(int(iters), ctypes.byref(out), _stream(stream))
    if st != 0:
        raise FAError(st, "fa_probe_ex2_rate")
    return out.value


def fa_set_wait_limit_ns(limit_ns):
    lib().fa_set_wait_limit_ns(int(limit_ns))


def fa_get_last_device_error(stream=None):
    return lib().fa_get_last_device_error(_stream(stream))


def fa_selftest_wait_timeout(stream=None):
    return lib().fa_selftest_wait_timeout(_stream(stream))


def fa_selftest_tile(a, b, s_out, o_out, a_copy, stream=None):
    """One-tile check of the tensor-core building blocks: s_out = a b^T,
    o_out = round(s_out) b (float32), a_copy = a read back from its swizzled
    shared-memory tile.  a, b, a_copy: [128, D] bf16 or fp16; returns the
    status code."""
    for t in (a, b, s_out, o_out, a_copy):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("fa_selftest_tile wants contiguous CUDA tensors")
    if s_out.dtype != torch.float32 or o_out.dtype != torch.float32 or a_copy.dtype != a.dtype:
        raise ValueError("s_out and o_out must be float32, a_copy of a's dtype")
    D = a.shape[-1]
    if (a.dim() != 2 or tuple(a.shape) != (128, D) or b.shape != a.shape or a_copy.shape != a.shape
            or b.dtype != a.dtype or tuple(s_out.shape) != (128, 128) or tuple(o_out.shape) != (128, D)):
        raise ValueError("fa_selftest_tile wants a, b, a_copy [128, D], s_out [128, 128], o_out [128, D]")
    dt = _DT.get(a.dtype, FA_F32)
    return lib().fa_selftest_tile(_ptr(a), _ptr(b), _ptr(s_out), _ptr(o_out), _ptr(a_copy), D, dt, _stream(stream))


def fa_fwd(q, k, v, o, lse, causal, scale=None, cu_seqlens=None, max_seqlen=None, stream=None):
    """Enqueue the forward kernel: writes o (dtype of q) and lse (float32)."""
    _check(q, k, v, o, lse, cu_seqlens)
    B, H, N, D, T = _dims(q, cu_seqlens, max_seqlen)
    if lse.dtype != torch.float32:
        raise ValueError("lse must be float32")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    st = lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, D, scale, int(bool(causal)),
                      _ptr(cu_seqlens), T, _DT[q.dtype], _stream(stream))
    if st != 0:
        raise FAError(st, "fa_fwd")


def fa_bwd_workspace_size(q, cu_seqlens=None, max_seqlen=None):
    B, H, N, D, T = _dims(q, cu_seqlens, max_seqlen)
    return int(lib().fa_bwd_workspace_size(B, H, N, D, _ptr(cu_seqlens), T, _DT[q.dtype]))


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, causal, scale=None, cu_seqlens=None, max_seqlen=None,
           workspace=None, stream=None):
    """Enqueue the backward kernels: writes dq, dk, dv (dtype of q)."""
    _check(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens)
    B, H, N, D, T = _dims(q, cu_seqlens, max_seqlen)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if workspace is None:
        need = fa_bwd_workspace_size(q, cu_seqlens, max_seqlen)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                      B, H, N, D, scale, int(bool(causal)), _ptr(cu_seqlens), T, _DT[q.dtype],
                      _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if st != 0:
        raise FAError(st, "fa_bwd")


def fa_bwd_static_ws(q, k, v, o, lse, dout, dq, dk, dv, causal, scale=None, cu_seqlens=None, max_seqlen=None,
                     stream=None):
    """fa_bwd without a workspace argument: the library's own fixed device
    buffer (FA_BWD_STATIC_WS_BYTES, 16 MiB) serves as scratch, for callers
    that cannot allocate device memory.  Calls sharing a device must not
    overlap on the GPU; problems needing more scratch raise FAError
    (FA_ERR_WORKSPACE)."""
    _check(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens)
    B, H, N, D, T = _dims(q, cu_seqlens, max_seqlen)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    st = lib().fa_bwd_static_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                _ptr(dv), B, H, N, D, scale, int(bool(causal)), _ptr(cu_seqlens), T, _DT[q.dtype],
                                _stream(stream))
    if st != 0:
        err = FAError(st, "fa_bwd_static_ws")
        detail = lib().fa_last_error_detail().decode()
        if detail and detail not in str(err):
            err = FAError(st, f"fa_bwd_static_ws [{detail}]")
        raise err


STATIC_WS_BYTES = 16 << 20


def fa_fwd_dropout(q, k, v, o, lse, causal, p_drop, seed, offset=0, scale=None, cu_seqlens=None, max_seqlen=None,
                   stream=None):
    """fa_fwd with attention dropout: weights dropped with probability p_drop
    (decisions regenerated from seed and offset), kept ones scaled by
    1 / (1 - p_drop); lse is that of the undropped softmax."""
    _check(q, k, v, o, lse, cu_seqlens)
    B, H, N, D, T = _dims(q, cu_seqlens, max_seqlen)
    if lse.dtype != torch.float32:
        raise ValueError("lse must be float32")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    st = lib().fa_fwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, D, scale, int(bool(causal)),
                              _ptr(cu_seqlens), T, _DT[q.dtype], float(p_drop), int(seed), int(offset),
                              _stream(stream))
    if st != 0:
        raise FAError(st, "fa_fwd_dropout")


def fa_bwd_dropout(q, k, v, o, lse, dout, dq, dk, dv, causal, p_drop, seed, offset=0, scale=None, cu_seqlens=None,
                   max_seqlen=None, workspace=None, stream=None):
    """fa_bwd for a forward run by fa_fwd_dropout with the same p_drop, seed, offset."""
    _check(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens)
    B, H, N, D, T = _dims(q, cu_seqlens, max_seqlen)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if workspace is None:
        need = fa_bwd_workspace_size(q, cu_seqlens, max_seqlen)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = lib().fa_bwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                              B, H, N, D, scale, int(bool(causal)), _ptr(cu_seqlens), T, _DT[q.dtype], float(p_drop),
                              int(seed), int(offset), _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream))
    if st != 0:
        raise FAError(st, "fa_bwd_dropout")


def fa_bwd_deterministic(q, k, v, o, lse, dout, dq, dk, dv, causal, scale=None, cu_seqlens=None, max_seqlen=None,
                         p_drop=0.0, seed=0, offset=0, workspace=None, stream=None):
    """fa_bwd (or fa_bwd_dropout) with every sum in a fixed order: repeated
    calls give bit-identical gradients (dQ from a query-stationary kernel)."""
    _check(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens)
    B, H, N, D, T = _dims(q, cu_seqlens, max_seqlen)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if workspace is None:
        rows = (H * T) if cu_seqlens is not None else (B * H * N)
        workspace = torch.empty((rows * 4 + 255) // 256 * 256 + 256, dtype=torch.uint8, device=q.device)
    st = lib().fa_bwd_deterministic(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                    _ptr(dv), B, H, N, D, scale, int(bool(causal)), _ptr(cu_seqlens), T,
                                    _DT[q.dtype], float(p_drop), int(seed), int(offset), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    if st != 0:
        raise FAError(st, "fa_bwd_deterministic")


def fa_decode_workspace_size(q, k):
    """Bytes of scratch fa_decode needs for q [B, H, nq, D] against k [B, H, nk, D]."""
    B, H, nq, D = q.shape
    return int(lib().fa_decode_workspace_size(B, H, nq, k.shape[2], D, _DT[q.dtype]))


def fa_decode(q, k, v, o, lse, causal, scale=None, workspace=None, stream=None):
    """Enqueue a cached decoding step: q [B, H, nq, D] against the cache
    k, v [B, H, nk, D]; query i is at position nk - nq + i.  Writes o (dtype of
    q) and lse [B, H, nq] (float32)."""
    _check(q, k, v, o, lse)
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3]:
        raise ValueError("q must be [B, H, nq, D] and k, v [B, H, nk, D]")
    if lse.dtype != torch.float32:
        raise ValueError("lse must be float32")
    B, H, nq, D = q.shape
    nk = k.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need = fa_decode_workspace_size(q, k)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().fa_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, nq, nk, D, scale, int(bool(causal)),
                         _DT[q.dtype], _ptr(workspace), nbytes, _stream(stream))
    if st != 0:
        raise FAError(st, "fa_decode")


def decode(q, k, v, causal=True, scale=None, stream=None):
    """Allocating convenience wrapper around fa_decode: returns (o, lse)."""
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    fa_decode(q, k, v, o, lse, causal, scale, stream=stream)
    return o, lse


def forward(q, k, v, causal=False, scale=None, cu_seqlens=None, max_seqlen=None, stream=None):
    """(o, lse) for dense [B,H,N,D] or packed [H,T,D] inputs."""
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, causal, scale, cu_seqlens, max_seqlen, stream)
    return o, lse


def backward(q, k, v, o, lse, dout, causal=False, scale=None, cu_seqlens=None, max_seqlen=None,
             workspace=None, stream=None):
    """(dq, dk, dv) given the forward outputs and the upstream gradient."""
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, causal, scale, cu_seqlens, max_seqlen, workspace, stream)
    return dq, dk, dv


# ---- cached serving: the 8-bit cache and the decoding steps that read it ----

class Cache8(NamedTuple):
    """An 8-bit key/value cache: k, v [B, Hk, cap, D] e4m3 codes
    (torch.float8_e4m3fn) and k_exp, v_exp [B, Hk, cap] uint8, one exponent
    byte a row; value = code * 2^(exp - 127)."""
    k: torch.Tensor
    v: torch.Tensor
    k_exp: torch.Tensor
    v_exp: torch.Tensor


def cache_alloc(B, Hk, cap, D, device="cuda"):
    """An empty 8-bit cache (codes and exponents zero) for B sequences of at
    most cap rows and Hk key heads."""
    k, v = (torch.zeros(B, Hk, cap, D, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
    k_exp, v_exp = (torch.zeros(B, Hk, cap, dtype=torch.uint8, device=device) for _ in range(2))
    return Cache8(k, v, k_exp, v_exp)


# A decoding step of a small batch takes the GPU a few microseconds, so these
# calls keep their own host cost down: one pass over the tensors, the stream's
# handle straight from torch (torch.cuda.current_stream builds an object, 3 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _elsewhere(t, stream):
    """Whether a call on t has to make another device or stream current first;
    refuses tensors that are not on a GPU."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    return stream is not None or t.get_device() != torch.cuda.current_device()


@contextlib.contextmanager
def _on(t, stream):
    """Makes t's device and `stream` (None: that device's current one) current
    for a call, so that its scratch and outputs are allocated for the stream
    that writes them."""
    with torch.cuda.device(t.device):
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream), device=t.device)
        with torch.cuda.stream(stream):
            yield


def _together(device, tensors):
    for t in tensors:
        if t is not None and (t.get_device() != device or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on one device")


def _check_cache8(k, v, k_exp, v_exp):
    if k.dim() != 4 or v.shape != k.shape or k_exp.shape != k.shape[:3] or v_exp.shape != k_exp.shape:
        raise ValueError("a cache holds k, v [B, Hk, cap, D] and k_exp, v_exp [B, Hk, cap]")
    if k.dtype != torch.float8_e4m3fn or v.dtype != torch.float8_e4m3fn:
        raise ValueError("cache codes must be float8_e4m3fn")
    if k_exp.dtype != torch.uint8 or v_exp.dtype != torch.uint8:
        raise ValueError("cache exponents must be uint8")


def _check_int32(name, t, B):
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != B:
        raise ValueError(f"{name} must be int32 [{B}]")


def _rows_call(where, k, v, cache, start, count, stream):
    kc, vc, ke, ve = cache
    if _elsewhere(k, stream):
        with _on(k, stream):
            return _rows_call(where, k, v, cache, start, count, None)
    device = k.get_device()
    _together(device, (k, v, kc, vc, ke, ve, start, count))
    _check_cache8(kc, vc, ke, ve)
    B, H, cap, D = kc.shape
    if k.dim() != 4 or v.shape != k.shape or (k.shape[0], k.shape[1], k.shape[3]) != (B, H, D):
        raise ValueError("k and v must be [B, Hk, n, D] with the cache's B, Hk and D")
    dt = _DT.get(k.dtype)
    if dt is None or v.dtype != k.dtype:
        raise ValueError("k and v must be both bfloat16, float16 or float32")
    at_start = at_count = None
    if start is not None:
        _check_int32("start", start, B)
        at_start = start.data_ptr()
    if count is not None:
        _check_int32("count", count, B)
        at_count = count.data_ptr()
    dense = (k.data_ptr(), v.data_ptr())
    held = (kc.data_ptr(), vc.data_ptr(), ke.data_ptr(), ve.data_ptr())
    st = getattr(lib(), where)(*(dense + held if where == "fa_cache_write" else held + dense), B, H, k.shape[2], cap, D,
                               at_start, at_count, dt, _raw_stream(device))
    if st != 0:
        raise FAError(st, where)


def fa_cache_write(k, v, cache, start=None, count=None, stream=None):
    """Quantise new rows k, v [B, Hk, n, D] (bf16, fp16 or fp32) into the 8-bit
    cache at rows start[b] .. start[b] + count[b] - 1 of every sequence (start,
    count: int32 [B] on the device; None: 0 and n).  Rows that are not
    addressed keep what they hold; a sequence whose range does not fit in the
    cache is skipped and reported by fa_get_last_device_error."""
    _rows_call("fa_cache_write", k, v, cache, start, count, stream)


def fa_cache_read(cache, k, v, start=None, count=None, stream=None):
    """Read rows start[b] .. start[b] + count[b] - 1 of the 8-bit cache into k,
    v [B, Hk, n, D] (bf16, fp16 or fp32); the rows after them become zeros."""
    _rows_call("fa_cache_read", k, v, cache, start, count, stream)


def cache_read(cache, start, n, count=None, dtype=torch.bfloat16, stream=None):
    """Allocating wrapper around fa_cache_read: returns (k, v) [B, Hk, n, D]."""
    held = cache[0]
    if _elsewhere(held, stream):
        with _on(held, stream):
            return cache_read(cache, start, n, count, dtype)
    B, H, _, D = held.shape
    k, v = (torch.empty((B, H, n, D), dtype=dtype, device=held.device) for _ in range(2))
    _rows_call("fa_cache_read", k, v, cache, start, count, None)
    return k, v


def _serve_dims(q, held, max_len):
    """(B, H, Hk, nq, cap, max_len, D) of a decoding step over a cache."""
    if q.dim() != 4 or held.dim() != 4:
        raise ValueError("q must be [B, H, nq, D] and the cache [B, Hk, cap, D]")
    B, H, nq, D = q.shape
    Bk, Hk, cap, Dk = held.shape
    if Bk != B or Dk != D or Hk == 0 or H % Hk:
        raise ValueError("q [B, H, nq, D] needs a cache [B, Hk, cap, D] with H a multiple of Hk")
    if max_len is None:
        return B, H, Hk, nq, cap, cap, D
    max_len = int(max_len)
    if not 0 <= max_len <= cap:
        raise ValueError("max_len must be between 0 and the cache's capacity")
    return B, H, Hk, nq, cap, max_len, D


def _serve_call(where, q, prefix, cache, lens, o, lse, causal, scale, max_len, workspace, stream):
    """The decoding steps over a cache; allocates what is None, returns (o, lse)."""
    B, H, Hk, nq, cap, max_len, D = _serve_dims(q, cache[0], max_len)
    dtype = q.dtype
    if len(cache) == 4:
        _check_cache8(*cache)
        held = tuple([t.data_ptr() for t in cache])
    elif len(cache) == 2 and cache[1].shape == cache[0].shape and cache[0].dtype == cache[1].dtype == dtype:
        held = (cache[0].data_ptr(), cache[1].data_ptr(), None, None)
    else:
        raise ValueError("the cache must be a Cache8, or a pair k, v [B, Hk, cap, D] of q's dtype")
    if _elsewhere(q, stream):
        with _on(q, stream):
            return _serve_call(where, q, prefix, cache, lens, o, lse, causal, scale, max_len, workspace, None)
    device = q.get_device()
    dt = _DT.get(dtype)
    if dt is None:
        raise ValueError("q must be bfloat16 or float16")
    if o is None:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, nq), dtype=torch.float32, device=q.device)
    else:
        if o.dtype != dtype or o.shape != q.shape:
            raise ValueError("o must have q's shape and dtype")
        if lse.dtype != torch.float32 or lse.shape != q.shape[:-1]:
            raise ValueError("lse must be float32 [B, H, nq]")
        _together(device, (o, lse, workspace))
    _together(device, (q, lens, *cache, *prefix))
    at_lens = None
    if lens is not None:
        _check_int32("lens", lens, B)
        at_lens = lens.data_ptr()
    n_prefix = 0
    if prefix:
        kp, vp = prefix
        if kp.dim() != 3 or vp.shape != kp.shape or kp.shape[0] != Hk or kp.shape[2] != D:
            raise ValueError("the prefix must be k, v [Hk, np, D]")
        if kp.dtype != dtype or vp.dtype != dtype:
            raise ValueError("the prefix must have q's dtype")
        n_prefix = kp.shape[1]
        head = (q.data_ptr(), kp.data_ptr(), vp.data_ptr())
        sizes = (B, H, Hk, nq, n_prefix, cap, max_len, D)
    else:
        head = (q.data_ptr(),)
        sizes = (B, H, Hk, nq, cap, max_len, D)
    library = lib()
    if workspace is None:
        nbytes = library.fa_decode_shared_workspace_size(B, H, Hk, nq, n_prefix, max_len, D, dt)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    st = getattr(library, where)(*head, *held, o.data_ptr(), lse.data_ptr(), *sizes,
                                 1.0 / math.sqrt(D) if scale is None else float(scale), 1 if causal else 0, at_lens, dt,
                                 workspace.data_ptr(), nbytes, _raw_stream(device))
    if st != 0:
        raise FAError(st, where)
    return o, lse


def fa_decode_cache_workspace_size(q, cache, max_len=None):
    """Bytes of scratch fa_decode_cache needs for q [B, H, nq, D] and this cache."""
    B, H, Hk, nq, _, max_len, D = _serve_dims(q, cache[0], max_len)
    return int(lib().fa_decode_cache_workspace_size(B, H, Hk, nq, max_len, D, _DT[q.dtype]))


def fa_decode_cache(q, cache, lens, o, lse, causal, scale=None, max_len=None, workspace=None, stream=None):
    """Enqueue a decoding step over an 8-bit cache: the new queries q [B, H, nq,
    D] (bf16 or fp16) against the first lens[b] rows (int32 [B] on the device;
    None: max_len) of each sequence, the new tokens' rows among them.  H must be
    a multiple of the cache's Hk; query head h reads key head h // (H // Hk).
    Query i is at position lens[b] - nq + i.  max_len (default: the capacity)
    bounds lens; the scratch and the work are laid out by it.  Writes o (dtype of q) and lse [B, H, nq] (float32); rows that
    see no key get 0 and -inf."""
    if len(cache) != 4:
        raise ValueError("the cache must be a Cache8")
    _serve_call("fa_decode_cache", q, (), cache, lens, o, lse, causal, scale, max_len, workspace, stream)


def decode_cache(q, cache, lens=None, causal=True, scale=None, max_len=None, stream=None):
    """Allocating wrapper around fa_decode_cache: returns (o, lse)."""
    if len(cache) != 4:
        raise ValueError("the cache must be a Cache8")
    return _serve_call("fa_decode_cache", q, (), cache, lens, None, None, causal, scale, max_len, None, stream)


def fa_decode_shared_workspace_size(q, k_prefix, cache, max_len=None):
    """Bytes of scratch fa_decode_shared needs for q [B, H, nq, D], a prefix
    k_prefix [Hk, np, D] and the sequences' own cache."""
    B, H, Hk, nq, _, max_len, D = _serve_dims(q, cache[0], max_len)
    return int(lib().fa_decode_shared_workspace_size(B, H, Hk, nq, k_prefix.shape[1], max_len, D, _DT[q.dtype]))


def fa_decode_shared(q, k_prefix, v_prefix, cache, lens, o, lse, causal, scale=None, max_len=None, workspace=None,
                     stream=None):
    """Enqueue a decoding step of a batch whose sequences share their first np
    keys: k_prefix, v_prefix [Hk, np, D] (dtype of q), then lens[b] rows of
    each sequence's own, in `cache`: a Cache8, or a pair k, v [B, Hk, cap, D] of
    q's dtype.  Query i is at position np + lens[b] - nq + i.  Everything else
    as for fa_decode_cache.  Give max_len where the cache is much longer than its
    sequences are: the SMs are shared out between prefix and own rows by it."""
    _serve_call("fa_decode_shared", q, (k_prefix, v_prefix), cache, lens, o, lse, causal, scale, max_len,
                workspace, stream)


def decode_shared(q, k_prefix, v_prefix, cache, lens=None, causal=True, scale=None, max_len=None, stream=None):
    """Allocating wrapper around fa_decode_shared: returns (o, lse)."""
    return _serve_call("fa_decode_shared", q, (k_prefix, v_prefix), cache, lens, None, None, causal, scale, max_len,
                       None, stream)
