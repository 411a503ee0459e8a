"""ctypes binding of libflashsample (include/flashsample.h).

Argument marshalling only: every step of sampling runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  If the
library is missing, or a tensor is not on a CUDA device, the call raises --
there is no CPU fallback.
"""

import ctypes
import os
from array import array
from functools import lru_cache
from operator import attrgetter

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libflashsample.so")

FS_OK = 0
FS_CHUNK_FIRST = 1
FS_CHUNK_LAST = 2
FS_CHUNK_SERIAL = 4
FS_PATH_AUTO, FS_PATH_SIMT, FS_PATH_TC_VOCAB, FS_PATH_TC_BATCH, FS_PATH_TC_PAIR = 0, 1, 2, 3, 4
FS_FAULT_NONE, FS_FAULT_ALLOC, FS_FAULT_LAUNCH, FS_FAULT_LATER_LAUNCH = 0, 1, 2, 3
FS_MEAN_TOKEN, FS_MEAN_SEQUENCE, FS_MEAN_NONE = 0, 1, 2
FS_TYPE_F32, FS_TYPE_BF16, FS_TYPE_F16 = 0, 1, 2
FS_TYPE_E4M3, FS_TYPE_E5M2 = 3, 4
FS_NORM_L2, FS_NORM_MAX = 0, 1
FS_SMALL_WORKSPACE = 524288

_c_void_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_u64 = ctypes.c_uint64
_int = ctypes.c_int

# name -> (restype, argtypes); mirrors include/flashsample.h
SIGNATURES = {
    "fs_sample": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _u64, _u64,
                         _c_void_p, _c_void_p, _c_void_p]),
    "fs_sample_ex": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _i64,
                            _u64, _u64, _c_void_p, _c_void_p, _c_void_p]),
    "fs_sample_chunked": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _i64, _c_void_p,
                                 _c_void_p, _i64, _u64, _u64, _c_void_p, _c_void_p, _int,
                                 _c_void_p, _c_void_p, _c_void_p]),
    "fs_sample_chunked_early": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _i64, _c_void_p,
                                       _c_void_p, _i64, _u64, _u64, _c_void_p, _c_void_p, _int,
                                       _c_void_p, ctypes.c_float, ctypes.c_float, _c_void_p,
                                       _c_void_p, _c_void_p, _c_void_p]),
    "fs_row_norms": (_int, [_c_void_p, _i64, _i64, _c_void_p, _c_void_p]),
    "fs_chunk_rest_norms": (_int, [_c_void_p, _i64, _c_void_p, _i64, _c_void_p, _c_void_p]),
    "fs_combine_shards": (_int, [_c_void_p, _c_void_p, _i64, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "fs_sample_topk": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _i64,
                              _u64, _u64, _int, _c_void_p, _c_void_p, _c_void_p]),
    "fs_sample_unfused": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _i64,
                                 _u64, _u64, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "fs_sample_host": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _i64,
                              _u64, _u64, _c_void_p, _c_void_p, _c_void_p]),
    "fs_sample_noalloc": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _u64, _u64,
                                 _c_void_p, _c_void_p, _c_void_p]),
    "fs_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "fs_workspace_reserve": (_int, [_i64, _i64, _c_void_p]),
    "fs_workspace_release": (_int, []),
    "fs_set_path": (_int, [_int]),
    "fs_set_launch_overlap": (_int, [_int]),
    "fs_path_for_batch": (_int, [_i64]),
    "fs_sample_chunked_step": (_int, [_c_void_p, _c_void_p, _i64, _i64, _c_void_p, _int, _c_void_p, _c_void_p,
                                      _i64, _u64, _u64, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                      _c_void_p]),
    "fs_path_for_chunks": (_int, [_i64, _i64, _int]),
    "fs_profile_events": (_int, [_c_void_p, _c_void_p]),
    "fs_device_error": (_int, [ctypes.POINTER(_int)]),
    "fs_debug_wait_timeout": (_int, [_u64, _c_void_p]),
    "fs_debug_set_fault": (_int, [_int]),
    "fs_status_string": (ctypes.c_char_p, [_int]),
    "fs_last_error": (ctypes.c_char_p, []),
    "fs_token_logprobs": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _i64,
                                 _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_size_t, _c_void_p]),
    "fs_token_logprobs_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "fs_logprob_buffer_elems": (_i64, [_i64, _i64]),
    "fs_token_logprobs_backward": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p,
                                          _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                          _c_void_p, ctypes.c_size_t, _c_void_p]),
    "fs_token_logprobs_backward_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "fs_policy_loss": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _i64, _i64,
                              ctypes.c_double, ctypes.c_double, ctypes.c_double, _int, _c_void_p, _c_void_p,
                              _c_void_p, ctypes.c_size_t, _c_void_p]),
    "fs_policy_loss_workspace_bytes": (ctypes.c_size_t, [_i64]),
    "fs_clip_grad_norm": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _int, ctypes.c_double, _int, _c_void_p,
                                 _c_void_p]),
    "fs_quantize_fp8": (_int, [_c_void_p, _int, _i64, _i64, _i64, _int, _int, _int, _c_void_p, _i64, _c_void_p, _i64,
                               _i64, _c_void_p]),
    "fs_fp8_matmul": (_int, [_c_void_p, _int, _i64, _c_void_p, _i64, _i64, _c_void_p, _int, _i64, _c_void_p, _i64, _i64,
                             _int, _i64, _i64, _i64, _c_void_p, _int, _i64, _c_void_p]),
    "fs_sample_fp8": (_int, [_c_void_p, _i64, _c_void_p, _i64, _i64, _c_void_p, _i64, _c_void_p, _i64, _i64, _int, _i64,
                             _i64, _i64, _c_void_p, _c_void_p, _i64, _u64, _u64, _c_void_p, _c_void_p, _c_void_p]),
    "fs_layer_norm": (_int, [_c_void_p, _int, _i64, _i64, _i64, _c_void_p, _c_void_p, _int, _int, ctypes.c_double,
                             _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _int, _i64, _c_void_p, _i64, _i64,
                             _c_void_p]),
    "fs_layer_norm_backward": (_int, [_c_void_p, _i64, _c_void_p, _int, _i64, _i64, _i64, _c_void_p, _int, _int,
                                      _c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p,
                                      ctypes.c_size_t, _c_void_p]),
    "fs_layer_norm_backward_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "fs_debug_noise": (_int, [_u64, _u64, _i64, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "fs_debug_fused_logits": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _i64,
                                     _u64, _u64, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
}


class FlashSampleError(RuntimeError):
    """A libflashsample call returned a non-OK status (or the library is missing)."""

    def __init__(self, status, detail):
        self.status = status
        super().__init__(f"{status}: {detail}")


_lib = None


def library():
    """Load libflashsample.so (once) and declare its signatures."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FlashSampleError("NOT_BUILT", f"{LIB_PATH} is missing; build it with "
                                   "`python -m lm_head_exact_gb300.build` (there is no CPU fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def check(status):
    if status != FS_OK:
        lib = library()
        raise FlashSampleError(lib.fs_status_string(status).decode(), lib.fs_last_error().decode())


def _torch():
    import torch
    return torch


def _stream_ptr(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name, dtype=None, ndim=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be a CUDA tensor (no CPU fallback)")
    if dtype is not None and t.dtype != dtype:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must have {ndim} dims")
    if not t.is_contiguous():
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _bias_args(bias, B, V):
    if bias is None:
        return ctypes.c_void_p(0), 0
    torch = _torch()
    if isinstance(bias, torch.Tensor) and bias.dim() == 2 and bias.stride(1) == 1:
        # a column slice of a [B, V] bias keeps its row stride
        if not bias.is_cuda or bias.dtype != torch.float32:
            raise FlashSampleError("FS_ERR_INVALID_ARG", "bias must be a float32 CUDA tensor (no CPU fallback)")
        return ctypes.c_void_p(bias.data_ptr()), bias.stride(0)
    ptr = _dev(bias, "bias", torch.float32, 1)
    return ptr, 0


def _made_on(stream, device, make):
    """The tensors that make() allocates, for a call that writes them on
    ``stream``: from that stream's memory, for what the current stream frees
    may still be in use there.  They are marked as used on the current stream,
    where the caller reads them once it has waited for ``stream``."""
    torch = _torch()
    if stream is None or torch.device(device).type != "cuda":  # (tensors elsewhere are refused by the call's checks)
        return make()
    current = torch.cuda.current_stream(device)
    if stream == current:
        return make()
    with torch.cuda.stream(stream):
        made = make()
    for t in made:
        t.record_stream(current)
    return made


def _outs(B, device, out, stream):
    torch = _torch()
    if out is not None:
        return out
    return _made_on(stream, device, lambda: (torch.empty(B, dtype=torch.int64, device=device),
                                             torch.empty(B, dtype=torch.float32, device=device)))


def sample(h, W, temp, seed, step, bias=None, out=None, stream=None):
    """Fused LM-head exact sample of one decode step.

    h: bf16 [B, d], W: bf16 [V, d], temp: fp32 [B] (CUDA tensors); bias:
    optional fp32 [B, V] or [V].  Returns (ids int64 [B], max fp32 [B]) on
    the device, enqueued on the current stream.
    """
    torch = _torch()
    B, d = h.shape
    V = W.shape[0]
    ids, mx = _outs(B, h.device, out, stream)
    bptr, bstride = _bias_args(bias, B, V)
    check(library().fs_sample_ex(_dev(h, "h", torch.bfloat16, 2), _dev(W, "W", torch.bfloat16, 2),
                                 B, d, V, _dev(temp, "temp", torch.float32, 1), bptr, bstride,
                                 seed, step, _dev(ids, "out_ids", torch.int64),
                                 _dev(mx, "out_max", torch.float32), _stream_ptr(stream)))
    return ids, mx


def debug_fused_logits(h, W, temp, seed, step, bias=None, stream=None):
    """``sample`` with the fused kernel's logit inspection store switched on:
    returns (ids, max, logits fp32 [B, V]), the logits being the values the
    fused kernel's epilogue read (accumulator + bias, before temperature and
    noise).  Same kernel family, instantiation and launch as ``sample``."""
    torch = _torch()
    B, d = h.shape
    V = W.shape[0]
    ids, mx = _outs(B, h.device, None, stream)
    logits, = _made_on(stream, h.device, lambda: (torch.full((B, V), float("nan"), dtype=torch.float32,
                                                             device=h.device),))
    bptr, bstride = _bias_args(bias, B, V)
    check(library().fs_debug_fused_logits(_dev(h, "h", torch.bfloat16, 2), _dev(W, "W", torch.bfloat16, 2),
                                          B, d, V, _dev(temp, "temp", torch.float32, 1), bptr, bstride,
                                          seed, step, _dev(ids, "out_ids", torch.int64),
                                          _dev(mx, "out_max", torch.float32), _dev(logits, "logits_out"),
                                          _stream_ptr(stream)))
    return ids, mx, logits


def sample_unfused(h, W, temp, seed, step, bias=None, logits_out=None, out=None, stream=None):
    """The unfused comparison pipeline (GEMM -> fp32 logits in HBM -> softmax
    -> sample).  Same inputs / outputs as ``sample``; ``logits_out`` (fp32
    [B, V] CUDA tensor) receives the logits if given."""
    torch = _torch()
    B, d = h.shape
    V = W.shape[0]
    ids, mx = _outs(B, h.device, out, stream)
    bptr, bstride = _bias_args(bias, B, V)
    lptr = _dev(logits_out, "logits_out", torch.float32) if logits_out is not None else ctypes.c_void_p(0)
    check(library().fs_sample_unfused(_dev(h, "h", torch.bfloat16, 2), _dev(W, "W", torch.bfloat16, 2),
                                      B, d, V, _dev(temp, "temp", torch.float32, 1), bptr, bstride,
                                      seed, step, _dev(ids, "out_ids", torch.int64),
                                      _dev(mx, "out_max", torch.float32), lptr, _stream_ptr(stream)))
    return ids, mx


def sample_ex(*args, **kwargs):
    """Alias of ``sample`` (the bias argument maps to fs_sample_ex)."""
    return sample(*args, **kwargs)


def combine_shards(shard_max, shard_ids, out=None, stream=None):
    """Tensor-parallel final step: per row, the best of the R shards' (max,
    id) pairs (shard_max fp32 [R, B], shard_ids int64 [R, B], device).
    Returns (ids int64 [B], max fp32 [B])."""
    torch = _torch()
    R, B = shard_max.shape
    ids, mx = _outs(B, shard_max.device, out, stream)
    check(library().fs_combine_shards(
        _dev(shard_max, "shard_max", torch.float32, 2), _dev(shard_ids, "shard_ids", torch.int64, 2), R, B,
        _dev(ids, "out_ids"), _dev(mx, "out_max"), _stream_ptr(stream)))
    return ids, mx


def tp_exchange(local_max, local_ids, group=None):
    """Exchange each rank's per-row (max, id) with the other ranks of
    ``group``: 8 bytes per row per rank (the fp32 max's bits and the id as
    int32), one all_gather.  Returns (all_max fp32 [R, B], all_ids int64
    [R, B]) on the inputs' device.  Communication plumbing only (NCCL for CUDA
    tensors, gloo for host tensors); the sample itself is computed by the
    library's kernels."""
    torch = _torch()
    import torch.distributed as dist
    R = dist.get_world_size(group)
    packed = torch.stack([local_max.contiguous().view(torch.int32), local_ids.to(torch.int32)], dim=1)
    parts = [torch.empty_like(packed) for _ in range(R)]
    dist.all_gather(parts, packed, group=group)
    allp = torch.stack(parts)
    return allp[..., 0].contiguous().view(torch.float32), allp[..., 1].to(torch.int64)


def sample_tp(h, W_shard, v_begin, temp, seed, step, group=None, bias_shard=None, stream=None):
    """Tensor-parallel sample: this rank holds vocabulary rows [v_begin,
    v_begin + W_shard.shape[0]); it samples its shard with global ids, the
    ranks exchange the per-row (max, id) pairs, and the combine picks the
    winner.  Every rank returns the same (ids, max), equal to sample() over
    the whole vocabulary."""
    torch = _torch()
    B = h.shape[0]
    out = _outs(B, h.device, None, stream)
    with torch.cuda.stream(stream):                        # (None: the current one) the exchange follows the sample
        cm = torch.empty(B, dtype=torch.float32, device=h.device)
        ci = torch.empty(B, dtype=torch.int64, device=h.device)
        local = sample_chunked(h, W_shard, v_begin, temp, seed, step, cm, ci, True, True, bias_chunk=bias_shard)
        all_max, all_ids = tp_exchange(local[1], local[0], group=group)
        return combine_shards(all_max, all_ids, out=out)


def sample_topk(h, W, temp, seed, step, k, bias=None, out=None, stream=None):
    """Gumbel-top-k: k ids per row without replacement, best first.
    Returns (ids int64 [B, k], z fp32 [B, k]); -1 / -inf where a row has
    fewer than k choosable ids.  1 <= k <= 16, B <= 4096; k = 1 gives
    sample()'s ids and maxima."""
    torch = _torch()
    B, d = h.shape
    V = W.shape[0]
    if out is None:
        out = _made_on(stream, h.device, lambda: (torch.empty((B, k), dtype=torch.int64, device=h.device),
                                                  torch.empty((B, k), dtype=torch.float32, device=h.device)))
    ids, z = out
    bptr, bstride = _bias_args(bias, B, V)
    check(library().fs_sample_topk(
        _dev(h, "h", torch.bfloat16, 2), _dev(W, "W", torch.bfloat16, 2), B, d, V,
        _dev(temp, "temp", torch.float32, 1), bptr, bstride, seed, step, int(k),
        _dev(ids, "out_ids", torch.int64, 2), _dev(z, "out_z", torch.float32, 2), _stream_ptr(stream)))
    return ids, z


def sample_chunked(h, W_chunk, v_begin, temp, seed, step, carry_max, carry_ids, first, last,
                   bias_chunk=None, out=None, stream=None, serial=False):
    """One chunk [v_begin, v_begin + W_chunk.shape[0]) of the grouped online
    variant; updates (carry_max, carry_ids) in place and, when ``last``,
    returns (ids, max)."""
    torch = _torch()
    B, d = h.shape
    v_end = v_begin + W_chunk.shape[0]
    flags = (FS_CHUNK_FIRST if first else 0) | (FS_CHUNK_LAST if last else 0) | (FS_CHUNK_SERIAL if serial else 0)
    ids = mx = None
    if last:
        ids, mx = _outs(B, h.device, out, stream)
    bptr, bstride = _bias_args(bias_chunk, B, W_chunk.shape[0])
    check(library().fs_sample_chunked(
        _dev(h, "h", torch.bfloat16, 2), _dev(W_chunk, "W_chunk", torch.bfloat16, 2), B, d,
        v_begin, v_end, _dev(temp, "temp", torch.float32, 1), bptr, bstride, seed, step,
        _dev(carry_max, "carry_max", torch.float32), _dev(carry_ids, "carry_ids", torch.int64),
        flags, _dev(ids, "out_ids") if last else ctypes.c_void_p(0),
        _dev(mx, "out_max") if last else ctypes.c_void_p(0), _stream_ptr(stream)))
    return (ids, mx) if last else None


def sample_chunked_step(h, W, bounds, temp, seed, step, carry_max, carry_ids, bias=None, out=None,
                        stream=None):
    """One whole chunked step over chunks [bounds[i], bounds[i+1]) of W in
    one C call (the per-chunk calls of ``sample_chunked`` issued from C).
    ``bounds`` may be a list or an int64 numpy array (kept by the caller to
    reuse).  Returns (ids, max)."""
    torch = _torch()
    B, d = h.shape
    b = bounds if isinstance(bounds, np.ndarray) and bounds.dtype == np.int64 else np.asarray(bounds, np.int64)
    n = len(b) - 1
    if n < 1 or b[-1] != W.shape[0]:
        raise FlashSampleError("FS_ERR_INVALID_ARG", "bounds must have >= 2 entries ending at W.shape[0]")
    ids, mx = _outs(B, h.device, out, stream)
    bptr, bstride = _bias_args(bias, B, W.shape[0])
    check(library().fs_sample_chunked_step(
        _dev(h, "h", torch.bfloat16, 2), _dev(W, "W", torch.bfloat16, 2), B, d, ctypes.c_void_p(b.ctypes.data), n,
        _dev(temp, "temp", torch.float32, 1), bptr, bstride, seed, step,
        _dev(carry_max, "carry_max", torch.float32), _dev(carry_ids, "carry_ids", torch.int64),
        _dev(ids, "out_ids"), _dev(mx, "out_max"), _stream_ptr(stream)))
    return ids, mx


def sample_chunked_early(h, W_chunk, v_begin, temp, seed, step, carry_max, carry_ids, first, last,
                         h_norms, rest_w_norm, rest_bias_max, done, bias_chunk=None, out=None, stream=None,
                         serial=False):
    """sample_chunked with online early finalization: ``h_norms`` fp32 [B]
    (row_norms(h)), ``rest_w_norm`` / ``rest_bias_max`` host floats bounding
    the later chunks, ``done`` a device int32 [1] flag: the first call
    resets it, a chunk sets it once every row's carried best can no longer be
    overtaken, and later calls that see it set skip their work.  ``serial``
    launches the call without overlapping the previous one."""
    torch = _torch()
    B, d = h.shape
    v_end = v_begin + W_chunk.shape[0]
    flags = (FS_CHUNK_FIRST if first else 0) | (FS_CHUNK_LAST if last else 0) | (FS_CHUNK_SERIAL if serial else 0)
    ids = mx = None
    if last:
        ids, mx = _outs(B, h.device, out, stream)
    bptr, bstride = _bias_args(bias_chunk, B, W_chunk.shape[0])
    check(library().fs_sample_chunked_early(
        _dev(h, "h", torch.bfloat16, 2), _dev(W_chunk, "W_chunk", torch.bfloat16, 2), B, d,
        v_begin, v_end, _dev(temp, "temp", torch.float32, 1), bptr, bstride, seed, step,
        _dev(carry_max, "carry_max", torch.float32), _dev(carry_ids, "carry_ids", torch.int64),
        flags, _dev(h_norms, "h_norms", torch.float32, 1), float(rest_w_norm), float(rest_bias_max),
        _dev(done, "done", torch.int32), _dev(ids, "out_ids") if last else ctypes.c_void_p(0),
        _dev(mx, "out_max") if last else ctypes.c_void_p(0), _stream_ptr(stream)))
    return (ids, mx) if last else None


def row_norms(X, out=None, stream=None):
    """fp32 Euclidean norms of the rows of a bf16 [n, d] device matrix."""
    torch = _torch()
    n, d = X.shape
    if out is None:
        out, = _made_on(stream, X.device, lambda: (torch.empty(n, dtype=torch.float32, device=X.device),))
    check(library().fs_row_norms(_dev(X, "X", torch.bfloat16, 2), n, d, _dev(out, "out", torch.float32, 1),
                                 _stream_ptr(stream)))
    return out


def chunk_rest_norms(W, bounds, stream=None):
    """Host list: for chunk i of ``bounds`` (n_chunks + 1 row offsets into W),
    the largest row norm of W after the chunk (0 for the last).  Synchronizes."""
    torch = _torch()
    b = np.ascontiguousarray(np.asarray(bounds, dtype=np.int64))
    n = len(b) - 1
    rest = np.zeros(max(n, 0), dtype=np.float32)
    check(library().fs_chunk_rest_norms(_dev(W, "W", torch.bfloat16, 2), W.shape[1],
                                        ctypes.c_void_p(b.ctypes.data), n,
                                        ctypes.c_void_p(rest.ctypes.data), _stream_ptr(stream)))
    return [float(x) for x in rest]


def sample_host(h_host, W, temp_host, seed, step, bias=None, out_ids=None, out_max=None,
                stream=None):
    """End-to-end call with host buffers (numpy arrays or CPU tensors; pinned
    memory recommended): h_host bf16 bits uint16 [B, d] (or a bf16 tensor),
    temp_host fp32 [B]; W (and bias) stay on the device.  Copies in, samples,
    copies out and synchronizes.  Returns host (ids int64 [B], max fp32 [B])."""
    torch = _torch()

    def host_ptr(a, name):
        if isinstance(a, np.ndarray):
            if not a.flags["C_CONTIGUOUS"]:
                raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be C-contiguous")
            return ctypes.c_void_p(a.ctypes.data)
        if isinstance(a, torch.Tensor) and not a.is_cuda and a.is_contiguous():
            return ctypes.c_void_p(a.data_ptr())
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be a contiguous host array")

    B, d = h_host.shape
    V = W.shape[0]
    if out_ids is None:
        out_ids = np.empty(B, dtype=np.int64)
    if out_max is None:
        out_max = np.empty(B, dtype=np.float32)
    bptr, bstride = _bias_args(bias, B, V)
    check(library().fs_sample_host(host_ptr(h_host, "h_host"), _dev(W, "W", torch.bfloat16, 2),
                                   B, d, V, host_ptr(temp_host, "temp_host"), bptr, bstride,
                                   seed, step, host_ptr(out_ids, "out_ids"),
                                   host_ptr(out_max, "out_max"), _stream_ptr(stream)))
    return out_ids, out_max


# ---------------------------------------------------------------- learning from sampled tokens
def _arg(t, name, dtype, shape=None):
    """Address of a contiguous CUDA tensor of this type and shape."""
    try:
        if t.is_cuda and t.dtype is dtype and (shape is None or t.shape == shape) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be a CUDA tensor (no CPU fallback)")
    if t.dtype != dtype:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be contiguous")


def _stream_of(t, stream):
    """Handle of ``stream``, or of the current stream of t's device (the raw
    handle: building a Stream object costs as much as the call itself)."""
    return stream.cuda_stream if stream is not None else _torch()._C._cuda_getCurrentRawStream(t.get_device())


def _head_args(h, W, ids, temp, bias):
    torch = _torch()
    try:
        (n, d), (V, d2) = h.shape, W.shape
    except (AttributeError, ValueError):
        d, d2 = 0, 1
    if d != d2:
        raise FlashSampleError("FS_ERR_INVALID_ARG", "h must be [n, d] and W [V, d]")
    bptr, bstride = None, 0
    if bias is not None:
        if tuple(bias.shape) not in ((n, V), (V,)):
            raise FlashSampleError("FS_ERR_INVALID_ARG", f"bias must be [n, V] or [V], got {tuple(bias.shape)}")
        bptr, bstride = _bias_args(bias, n, V)
    return (_arg(h, "h", torch.bfloat16), _arg(W, "W", torch.bfloat16), n, d, V,
            _arg(ids, "ids", torch.int64, (n,)), _arg(temp, "temp", torch.float32, (n,)), bptr, bstride)


# Bytes of workspace by sizes and the current device: the library lays it out
# for the pairs of SMs that the device holds at a time.
@lru_cache(maxsize=256)
def _forward_bytes(n, d, V, device):
    return library().fs_token_logprobs_workspace_bytes(n, d, V)


@lru_cache(maxsize=256)
def _backward_bytes(n, d, V, device):
    return library().fs_token_logprobs_backward_workspace_bytes(n, d, V)


@lru_cache(maxsize=256)
def _kept_elems(n, V):
    return library().fs_logprob_buffer_elems(n, V)


def _workspace(nbytes, device, stream):
    """(tensor, address) of device memory for one call, allocated on the
    stream that the call runs on: it may be handed out again as soon as the
    call returns, but only to work that follows on that stream.  Small ones
    come from the library's own block (NULL)."""
    if nbytes <= FS_SMALL_WORKSPACE:
        return None, None
    torch = _torch()
    if stream is None:
        t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        with torch.cuda.stream(stream):
            t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, t.data_ptr()


def logprob_buffer(n, V, device="cuda", stream=None):
    """The fp32 buffer in which ``token_logprobs`` leaves the logits of n rows
    for ``token_logprobs_backward``; ``stream``: the one that those calls are
    given, if not the current one."""
    torch = _torch()
    return _made_on(stream, device, lambda: (torch.empty(_kept_elems(n, V), dtype=torch.float32, device=device),))[0]


def _kept_arg(kept, n, V):
    torch = _torch()
    if kept is None:
        return None
    if kept.numel() != _kept_elems(n, V):
        raise FlashSampleError("FS_ERR_INVALID_ARG", "kept must be logprob_buffer(n, V)")
    return _arg(kept, "kept", torch.float32)


def token_logprobs(h, W, ids, temp, bias=None, kept=None, out=None, stream=None):
    """Log-probabilities of the tokens ``ids`` under softmax((h Wᵀ + bias) /
    temp), fused into the LM-head matmul.

    h: bf16 [n, d], W: bf16 [V, d], ids: int64 [n] (outside [0, V): the row is
    not scored, e.g. -1 for padding), temp: fp32 [n], bias: optional fp32
    [n, V] or [V].  ``kept`` (``logprob_buffer``) keeps the logits for the
    backward pass; without it they never reach device memory.  Returns
    (logp fp32 [n], lse fp32 [n])."""
    torch = _torch()
    args = _head_args(h, W, ids, temp, bias)
    n, d, V = args[2:5]
    if out is None:
        out = _made_on(stream, temp.device, lambda: (torch.empty_like(temp), torch.empty_like(temp)))
    logp, lse = out
    nbytes = _forward_bytes(n, d, V, torch.cuda.current_device())
    work, where = _workspace(nbytes, h.device, stream)
    check(library().fs_token_logprobs(
        *args, _arg(logp, "logp", torch.float32, (n,)), _arg(lse, "lse", torch.float32, (n,)), _kept_arg(kept, n, V),
        where, nbytes, _stream_of(h, stream)))
    return logp, lse


def token_logprobs_backward(h, W, ids, temp, logp, lse, grad_logp, bias=None, kept=None, need_h=True, need_W=True,
                            out=None, stream=None):
    """Gradients of ``token_logprobs``: from ``grad_logp`` (dL/dlogp, fp32
    [n]) to (grad_h bf16 [n, d], grad_W bf16 [V, d]); one that is not needed is
    None.  ``logp``, ``lse`` and ``kept`` are the forward call's (without
    ``kept`` the logits are formed again).  ``out``: the two tensors to
    write, where given."""
    torch = _torch()
    args = _head_args(h, W, ids, temp, bias)
    n, d, V = args[2:5]
    grad_h, grad_W = out if out is not None else (None, None)
    if need_h and grad_h is None:
        grad_h, = _made_on(stream, h.device, lambda: (torch.empty_like(h),))
    if need_W and grad_W is None:
        grad_W, = _made_on(stream, h.device, lambda: (torch.empty_like(W),))
    nbytes = _backward_bytes(n, d, V, torch.cuda.current_device())
    work, where = _workspace(nbytes, h.device, stream)
    check(library().fs_token_logprobs_backward(
        *args, _arg(logp, "logp", torch.float32, (n,)), _arg(lse, "lse", torch.float32, (n,)),
        _arg(grad_logp, "grad_logp", torch.float32, (n,)), _kept_arg(kept, n, V),
        _arg(grad_h, "grad_h", torch.bfloat16, (n, d)) if need_h else None,
        _arg(grad_W, "grad_W", torch.bfloat16, (V, d)) if need_W else None,
        where, nbytes, _stream_of(h, stream)))
    return grad_h if need_h else None, grad_W if need_W else None


_MEANS = {"token": FS_MEAN_TOKEN, "sequence": FS_MEAN_SEQUENCE, "none": FS_MEAN_NONE}


def policy_loss(logp, old_logp, advantages, seq_starts=None, mask=None, ref_logp=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0, mean="token", adv_per_seq=None, out=None, stream=None):
    """Clipped policy loss with a KL penalty against ``ref_logp``, and its
    gradient, in one call.

    ``logp``, ``old_logp`` and ``ref_logp``: fp32, either packed [N] with
    ``seq_starts`` (int64 [S + 1] on the device, from 0 to N) or padded
    [S, L]; [N] without ``seq_starts`` is one sequence.  ``advantages``: fp32
    [S], or one per token in logp's shape (``adv_per_seq`` says which where S
    = N packed tokens leave it open).  ``mask``: bool in logp's shape,
    False where a token takes no part.  ``mean``: "token", "sequence" or
    "none" (the sum).  Returns (stats fp32 [4]: loss, policy term, KL term,
    share of clipped tokens; grad fp32 in logp's shape = dloss/dlogp)."""
    torch = _torch()
    f32 = torch.float32
    ptr = _arg(logp, "logp", f32)
    shape = logp.shape
    if len(shape) not in (1, 2) or (len(shape) == 2 and seq_starts is not None):
        raise FlashSampleError("FS_ERR_INVALID_ARG", "logp must be [N], with or without seq_starts, or [S, L]")
    if mean not in _MEANS:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"mean must be one of {sorted(_MEANS)}, got {mean!r}")
    starts = None
    if seq_starts is not None:
        starts = _arg(seq_starts, "seq_starts", torch.int64)
        S = seq_starts.numel() - 1
        if seq_starts.dim() != 1 or S < 0:
            raise FlashSampleError("FS_ERR_INVALID_ARG", "seq_starts must be [S + 1]")
    else:
        S = shape[0] if len(shape) == 2 else 1
    N = logp.numel()
    if adv_per_seq is None:
        if seq_starts is not None and S == N and advantages.shape == shape:
            raise FlashSampleError("FS_ERR_INVALID_ARG", "as many sequences as tokens: say adv_per_seq")
        adv_per_seq = advantages.shape != shape
    adv = _arg(advantages, "advantages", f32, (S,) if adv_per_seq else shape)
    if out is None:
        out = _made_on(stream, logp.device,
                       lambda: (torch.empty(4, dtype=f32, device=logp.device), torch.empty_like(logp)))
    stats, grad = out
    lib = library()
    work, where, nbytes = None, None, 0
    if mean == "sequence":                    # one count for each sequence
        nbytes = lib.fs_policy_loss_workspace_bytes(S)
        work, where = _workspace(nbytes, logp.device, stream)
    check(lib.fs_policy_loss(
        ptr, _arg(old_logp, "old_logp", f32, shape), None if ref_logp is None else _arg(ref_logp, "ref_logp", f32, shape),
        adv, 1 if adv_per_seq else 0, None if mask is None else _arg(mask, "mask", torch.bool, shape), starts, S, N,
        clip_low, clip_high, kl_coef, _MEANS[mean], _arg(stats, "stats", f32, (4,)), _arg(grad, "grad", f32, shape),
        where, nbytes, _stream_of(logp, stream)))
    return stats, grad


_CLIP_TYPES = {}
_DTYPE = attrgetter("dtype")


def clip_grad_norm(grads, max_norm, out=None, norm_type=2.0, stream=None):
    """The norm of ``grads`` taken as one vector (fp32 scalar tensor, before
    scaling), and their scaling by min(1, max_norm / (norm + 1e-6)): in place,
    or into the tensors ``out``.  fp32, bf16 and fp16 tensors may be mixed;
    ``norm_type`` 2 or inf.  A norm that is not finite scales nothing; an
    infinite ``max_norm`` measures only.  Nothing is synchronized."""
    torch = _torch()
    if norm_type not in (2, float("inf")):
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"norm_type must be 2 or inf, got {norm_type}")
    if not _CLIP_TYPES:
        _CLIP_TYPES.update({torch.float32: FS_TYPE_F32, torch.bfloat16: FS_TYPE_BF16, torch.float16: FS_TYPE_F16})
    grads = list(grads)
    n = len(grads)
    tensor = torch.Tensor
    try:                                      # (maps: a dozen Python steps for each tensor cost more than the kernels)
        dtypes = list(map(_DTYPE, grads))
        types = array("i", map(_CLIP_TYPES.__getitem__, dtypes))
        fine = all(map(tensor.is_contiguous, grads)) and (n == 0 or grads[0].is_cuda)   # (the library checks each)
    except (AttributeError, KeyError, TypeError):
        fine = False
    if not fine:
        raise FlashSampleError("FS_ERR_INVALID_ARG", "gradients must be contiguous fp32, bf16 or fp16 CUDA tensors "
                               "(no CPU fallback)")
    pointers = outs = array("Q", map(tensor.data_ptr, grads))
    sizes = array("q", map(tensor.numel, grads))
    if out is not None:
        out = list(out)
        if len(out) != n:
            raise FlashSampleError("FS_ERR_INVALID_ARG", f"out must hold {n} tensors, got {len(out)}")
        if (list(map(_DTYPE, out)) != dtypes or array("q", map(tensor.numel, out)) != sizes
                or not all(map(tensor.is_contiguous, out))):
            raise FlashSampleError("FS_ERR_INVALID_ARG", "an output must be a contiguous CUDA tensor of its "
                                   "gradient's type and shape")
        outs = array("Q", map(tensor.data_ptr, out))
    device = grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
    norm, = _made_on(stream, device, lambda: (torch.empty((), dtype=torch.float32, device=device),))
    check(library().fs_clip_grad_norm(pointers.buffer_info()[0], outs.buffer_info()[0], sizes.buffer_info()[0],
                                      types.buffer_info()[0], n, max_norm,
                                      FS_NORM_L2 if norm_type == 2 else FS_NORM_MAX, norm.data_ptr(),
                                      _stream_of(norm, stream)))
    return norm


# ---------------------------------------------------------------- an 8-bit LM head and the norm ahead of it
_TYPES = {}


def _types():
    """FS_TYPE_* by torch type."""
    if not _TYPES:
        torch = _torch()
        _TYPES.update({torch.float32: FS_TYPE_F32, torch.bfloat16: FS_TYPE_BF16, torch.float16: FS_TYPE_F16,
                       torch.float8_e4m3fn: FS_TYPE_E4M3, torch.float8_e5m2: FS_TYPE_E5M2})
    return _TYPES


_WIDE = (FS_TYPE_F32, FS_TYPE_BF16, FS_TYPE_F16)
_FP8 = (FS_TYPE_E4M3, FS_TYPE_E5M2)


def _rows(t, name, types, shape=None):
    """(address, FS_TYPE_*, rows, columns, row stride) of a CUDA matrix of one
    of these types whose rows are contiguous."""
    try:
        kind = (_TYPES or _types()).get(t.dtype)
        rows, cols = t.shape
        if kind in types and t.is_cuda and (shape is None or (rows, cols) == shape):
            rs, cs = t.stride()
            if cs == 1 or cols <= 1:
                return t.data_ptr(), kind, rows, cols, rs if rows > 1 else max(rs, cols)
    except (AttributeError, ValueError):
        pass
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be a CUDA tensor (no CPU fallback)")
    if _types().get(t.dtype) not in types:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must not be {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be {'a matrix' if shape is None else tuple(shape)}, "
                               f"got {tuple(t.shape)}")
    raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must have contiguous rows")


def _fp8_rows(q, name, types, shape=None):
    """``_rows`` of an 8-bit matrix: the library wants rows that lie a multiple
    of 16 bytes apart, and a single row is as good as one."""
    at, kind, rows, cols, stride = _rows(q, name, types, shape)
    return at, kind, rows, cols, stride if rows > 1 else (stride + 15) // 16 * 16


def _scale_args(scale, name, rows, cols):
    """(address, row stride, column stride, rows of a block) of the scales of
    an 8-bit [rows, cols]."""
    cb = (cols + 127) // 128
    try:
        if scale.is_cuda and scale.dtype is _torch().float32:
            shape = scale.shape
            if shape == (rows, cb):
                return scale.data_ptr(), *scale.stride(), 1
            if shape == ((rows + 127) // 128, cb):
                return scale.data_ptr(), *scale.stride(), 128
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(scale, torch.Tensor) or not scale.is_cuda or scale.dtype != torch.float32:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be a float32 CUDA tensor (no CPU fallback)")
    raise FlashSampleError("FS_ERR_INVALID_ARG", f"{name} must be [{rows}, {cb}] or [{-(-rows // 128)}, {cb}], "
                           f"got {tuple(scale.shape)}")


def _fp8_out(rows, cols, block_rows, dtype, device, out, stream):
    """(q, scale, address, FS_TYPE_*, row stride, the scales' address and
    strides): ``out``, or new ones: rows of whole 16 bytes, and the scales of
    single rows side by side for a block, as the products read them fastest."""
    kind = (_TYPES or _types()).get(dtype)
    if kind not in _FP8:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"dtype must be float8_e4m3fn or float8_e5m2, got {dtype}")
    rb, cb = (rows if block_rows == 1 else (rows + 127) // 128), (cols + 127) // 128
    if out is not None:
        q, scale = out
        at, kind, _, _, stride = _fp8_rows(q, "q", _FP8, (rows, cols))
        s_at, s_row, s_col, _ = _scale_args(scale, "scale", rows, cols)
        if scale.shape[0] != rb:
            raise FlashSampleError("FS_ERR_INVALID_ARG", f"scale must have {rb} rows")
        return q, scale, at, kind, stride, s_at, s_row, s_col
    torch = _torch()
    stride = (cols + 15) // 16 * 16
    s_row, s_col = (1, rb) if block_rows == 1 else (cb, 1)
    if stream is None:
        q = torch.empty_strided((rows, cols), (stride, 1), dtype=dtype, device=device)
        scale = torch.empty_strided((rb, cb), (s_row, s_col), dtype=torch.float32, device=device)
    else:
        q, scale = _made_on(stream, device, lambda: (
            torch.empty_strided((rows, cols), (stride, 1), dtype=dtype, device=device),
            torch.empty_strided((rb, cb), (s_row, s_col), dtype=torch.float32, device=device)))
    return q, scale, q.data_ptr(), kind, stride, scale.data_ptr(), s_row, s_col


def _new(shape, dtype, device, stream):
    """A tensor for a call that writes it on ``stream``."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _made_on(stream, device, lambda: (torch.empty(shape, dtype=dtype, device=device),))[0]


def quantize_fp8(x, block_rows=1, dtype=None, transpose=False, out=None, stream=None):
    """x (fp32, bf16 or fp16 [r, c], contiguous rows), or with ``transpose``
    its transpose, in 8 bits with one fp32 scale for each block of block_rows
    (1 or 128) x 128 elements.

    ``dtype``: torch.float8_e4m3fn (default) or float8_e5m2.  Returns (q
    [R, C], scale [ceil(R / block_rows), ceil(C / 128)]); the value is q times
    its block's scale.  Rows of q lie a multiple of 16 bytes apart, so q is
    contiguous where C is one; the scales of single rows are a transposed
    view.  Hidden states are quantised by rows, weights in blocks of 128 x
    128 (``block_rows=128``), once."""
    ptr, kind, rows, cols, stride = _rows(x, "x", _WIDE)
    if block_rows not in (1, 128):
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"block_rows must be 1 or 128, got {block_rows}")
    R, C = (cols, rows) if transpose else (rows, cols)
    q, scale, *to = _fp8_out(R, C, block_rows, _torch().float8_e4m3fn if dtype is None else dtype, x.device, out, stream)
    q_ptr, q_kind, q_stride, s_ptr, s_row, s_col = to
    check(library().fs_quantize_fp8(ptr, kind, rows, cols, stride, 1 if transpose else 0, block_rows, q_kind, q_ptr, q_stride,
                                    s_ptr, s_row, s_col, _stream_of(x, stream)))
    return q, scale


def fp8_matmul(a, a_scale, b, b_scale, out_dtype=None, out=None, stream=None):
    """a bᵀ of two 8-bit matrices: a [m, k] quantised by rows, b [n, k] by rows
    or in blocks of 128 x 128 (told by the shape of its scales).  Returns
    [m, n] of ``out_dtype`` (bf16 by default; fp32 or fp16), or writes ``out``.
    (A result that becomes the W of ``sample``: some other work goes between
    the two calls, for ``sample`` reads W ahead, see fs_set_launch_overlap.)"""
    a_ptr, a_kind, m, k, a_stride = _fp8_rows(a, "a", _FP8)
    b_ptr, b_kind, n, k2, b_stride = _fp8_rows(b, "b", _FP8)
    if k != k2:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"a must be [m, k] and b [n, k], got {tuple(a.shape)} and {tuple(b.shape)}")
    as_ptr, as_row, as_col, _ = _scale_args(a_scale, "a_scale", m, k)
    if a_scale.shape[0] != m:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"a_scale must have a row for each of a's {m}")
    bs_ptr, bs_row, bs_col, block = _scale_args(b_scale, "b_scale", n, k)
    if out is None:
        out = _new((m, n), out_dtype or _torch().bfloat16, a.device, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"out must be {out_dtype}, got {out.dtype}")
    o_ptr, o_kind, _, _, o_stride = _rows(out, "out", _WIDE, (m, n))
    check(library().fs_fp8_matmul(a_ptr, a_kind, a_stride, as_ptr, as_row, as_col, b_ptr, b_kind, b_stride, bs_ptr, bs_row,
                                  bs_col, block, m, n, k, o_ptr, o_kind, o_stride, _stream_of(a, stream)))
    return out


def sample_fp8(h, h_scale, W, W_scale, temp, seed, step, bias=None, out=None, stream=None):
    """``sample`` with h [B, d] and the head W [V, d] in 8 bits (float8_e4m3fn):
    h quantised by rows (``quantize_fp8(h)``, ``layer_norm_fp8``), W by rows
    or in blocks of 128 x 128 (``quantize_fp8(W, block_rows=128)``, once).
    Reads half the bytes of a bf16 head.  Returns (ids int64 [B], max fp32 [B])."""
    torch = _torch()
    h_ptr, _, B, d, h_stride = _fp8_rows(h, "h", (FS_TYPE_E4M3,))
    W_ptr, _, V, d2, W_stride = _fp8_rows(W, "W", (FS_TYPE_E4M3,))
    if d != d2:
        raise FlashSampleError("FS_ERR_INVALID_ARG", "h must be [B, d] and W [V, d]")
    hs_ptr, hs_row, hs_col, _ = _scale_args(h_scale, "h_scale", B, d)
    if h_scale.shape[0] != B:
        raise FlashSampleError("FS_ERR_INVALID_ARG", f"h_scale must have a row for each of h's {B}")
    Ws_ptr, Ws_row, Ws_col, block = _scale_args(W_scale, "W_scale", V, d)
    bptr, bstride = None, 0
    if bias is not None:
        if tuple(bias.shape) not in ((B, V), (V,)):
            raise FlashSampleError("FS_ERR_INVALID_ARG", f"bias must be [B, V] or [V], got {tuple(bias.shape)}")
        bptr, bstride = _bias_args(bias, B, V)
    ids, mx = _outs(B, h.device, out, stream)
    check(library().fs_sample_fp8(h_ptr, h_stride, hs_ptr, hs_row, hs_col, W_ptr, W_stride, Ws_ptr, Ws_row, Ws_col, block,
                                  B, d, V, _arg(temp, "temp", torch.float32, (B,)), bptr, bstride, seed, step,
                                  _arg(ids, "out_ids", torch.int64, (B,)), _arg(mx, "out_max", torch.float32, (B,)),
                                  _stream_of(h, stream)))
    return ids, mx


def _norm_args(x, weight, bias):
    """x's ``_rows``, then the addresses and FS_TYPE_* of weight and bias:
    None, or [d] in one type, fp32 or x's."""
    ptr, kind, n, d, stride = _rows(x, "x", _WIDE)
    w = b = None
    w_kind = FS_TYPE_F32
    torch = _torch()
    if weight is not None:
        dtype = torch.float32 if getattr(weight, "dtype", None) is torch.float32 else x.dtype
        w, w_kind = _arg(weight, "weight", dtype, (d,)), _TYPES[dtype]
    if bias is not None:
        dtype = torch.float32 if getattr(bias, "dtype", None) is torch.float32 else x.dtype
        b = _arg(bias, "bias", dtype, (d,))
        if weight is not None and _TYPES[dtype] != w_kind:
            raise FlashSampleError("FS_ERR_INVALID_ARG", f"weight and bias must have one type, got {weight.dtype} and {bias.dtype}")
        w_kind = _TYPES[dtype]
    return ptr, kind, n, d, stride, w, b, w_kind


def layer_norm(x, weight=None, bias=None, eps=1e-5, rms=False, out=None, stream=None):
    """Layer norm of the rows of x (fp32, bf16 or fp16 [n, d], contiguous
    rows): (x - mean) rstd weight + bias; with ``rms`` without the mean.
    ``weight`` and ``bias`` [d]: fp32 or x's type, or None.  Returns (y, mean,
    rstd): y in x's type, the statistics fp32 [n] for ``layer_norm_backward``
    (mean is None with ``rms``).  ``out``: the tensor to write, x itself
    included.  d <= 32768.  (A result that becomes the W of ``sample``: as with
    ``fp8_matmul``.)"""
    torch = _torch()
    ptr, kind, n, d, stride, w, b, w_kind = _norm_args(x, weight, bias)
    device = x.device
    mean = None if rms else _new(n, torch.float32, device, stream)
    rstd = _new(n, torch.float32, device, stream)
    if out is None:
        out = _new((n, d), x.dtype, device, stream)
        y_ptr, y_stride = out.data_ptr(), d
    else:
        y_ptr, _, _, _, y_stride = _rows(out, "out", (kind,), (n, d))
    check(library().fs_layer_norm(ptr, kind, n, d, stride, w, b, w_kind, 1 if rms else 0, eps, y_ptr, y_stride,
                                  None if rms else mean.data_ptr(), rstd.data_ptr(), None, 0, 0, None, 0, 0,
                                  _stream_of(x, stream)))
    return out, mean, rstd


def layer_norm_fp8(x, weight=None, bias=None, eps=1e-5, rms=False, dtype=None, out=None, stream=None):
    """``layer_norm`` whose result is quantised by rows from its fp32 values, in
    the same pass: returns (q [n, d], scale [n, ceil(d / 128)]) as
    ``quantize_fp8`` does, for ``fp8_matmul`` and ``sample_fp8``."""
    ptr, kind, n, d, stride, w, b, w_kind = _norm_args(x, weight, bias)
    q, scale, *to = _fp8_out(n, d, 1, _torch().float8_e4m3fn if dtype is None else dtype, x.device, out, stream)
    q_ptr, q_kind, q_stride, s_ptr, s_row, s_col = to
    check(library().fs_layer_norm(ptr, kind, n, d, stride, w, b, w_kind, 1 if rms else 0, eps, None, 0, None, None, q_ptr,
                                  q_kind, q_stride, s_ptr, s_row, s_col, _stream_of(x, stream)))
    return q, scale


@lru_cache(maxsize=256)
def _norm_grad_bytes(n, d):
    return library().fs_layer_norm_backward_workspace_bytes(n, d)


def layer_norm_backward(grad, x, weight, mean, rstd, need_x=True, need_weight=True, need_bias=True, weight_dtype=None,
                        out=None, stream=None):
    """Gradients of ``layer_norm``: from ``grad`` (dL/dy, x's type [n, d]) to
    (grad_x in x's type, grad_weight and grad_bias [d] in the weight's type);
    one that is not needed is None.  ``mean`` and ``rstd`` are the forward
    call's; a ``mean`` of None says that it was called with ``rms``.
    ``weight_dtype``: the type of the two sums where weight is None (fp32).
    ``out``: the tensor for grad_x, ``grad`` or x itself included."""
    torch = _torch()
    x_ptr, kind, n, d, x_stride, w, _, w_kind = _norm_args(x, weight, None)
    g_ptr, _, _, _, g_stride = _rows(grad, "grad", (kind,), (n, d))
    if weight is None and weight_dtype is not None:
        w_kind = _TYPES.get(weight_dtype)
        if weight_dtype not in (torch.float32, x.dtype):
            raise FlashSampleError("FS_ERR_INVALID_ARG", f"weight_dtype must be float32 or {x.dtype}, got {weight_dtype}")
    w_dtype = torch.float32 if w_kind == FS_TYPE_F32 else x.dtype
    device, f32 = x.device, torch.float32
    gx_ptr, gx_stride, gx = None, 0, None
    if need_x:
        if out is None:
            gx = _new((n, d), x.dtype, device, stream)
            gx_ptr, gx_stride = gx.data_ptr(), d
        else:
            gx = out
            gx_ptr, _, _, _, gx_stride = _rows(gx, "out", (kind,), (n, d))
    gw = _new(d, w_dtype, device, stream) if need_weight else None
    gb = _new(d, w_dtype, device, stream) if need_bias else None
    nbytes = _norm_grad_bytes(n, d) if need_weight or need_bias else 0
    work, where = _workspace(nbytes, device, stream)
    check(library().fs_layer_norm_backward(
        g_ptr, g_stride, x_ptr, kind, n, d, x_stride, w, w_kind, 1 if mean is None else 0,
        None if mean is None else _arg(mean, "mean", f32, (n,)), _arg(rstd, "rstd", f32, (n,)), gx_ptr, gx_stride,
        None if gw is None else gw.data_ptr(), None if gb is None else gb.data_ptr(), where, nbytes, _stream_of(x, stream)))
    return gx, gw, gb


def debug_noise(seed, step, row0, n_rows, v0, n_vocab, stream=None):
    """(words uint32-as-int32 [n_rows, n_vocab], gumbel fp32 [n_rows, n_vocab])
    exactly as the sampling kernels draw them."""
    torch = _torch()
    words = torch.empty((n_rows, n_vocab), dtype=torch.int32, device="cuda")
    g = torch.empty((n_rows, n_vocab), dtype=torch.float32, device="cuda")
    check(library().fs_debug_noise(seed, step, row0, n_rows, v0, n_vocab,
                                   ctypes.c_void_p(words.data_ptr()), ctypes.c_void_p(g.data_ptr()),
                                   _stream_ptr(stream)))
    return words, g


def set_path(path):
    check(library().fs_set_path(path))


def debug_set_fault(kind):
    """Host-side fault injection (FS_FAULT_NONE / _ALLOC / _LAUNCH)."""
    check(library().fs_debug_set_fault(int(kind)))


def set_launch_overlap(enable):
    """Overlapped (programmatic dependent) launch of one-shot calls: True by
    default; False where the kernel enqueued just before a call may write W."""
    check(library().fs_set_launch_overlap(1 if enable else 0))


def path_for_batch(B):
    return library().fs_path_for_batch(B)


def path_for_chunks(B, V_chunk, step_chunks):
    return library().fs_path_for_chunks(B, V_chunk, step_chunks)


def workspace_reserve(B, V, stream=None):
    check(library().fs_workspace_reserve(B, V, _stream_ptr(stream)))


def profile_events(start, stop):
    """Record torch.cuda.Event ``start``/``stop`` around the fused kernel of
    every later call on this thread (None, None to stop)."""
    if start is None:
        check(library().fs_profile_events(None, None))
    else:
        check(library().fs_profile_events(ctypes.c_void_p(start.cuda_event),
                                          ctypes.c_void_p(stop.cuda_event)))


def debug_wait_timeout(timeout_ns, stream=None):
    check(library().fs_debug_wait_timeout(timeout_ns, _stream_ptr(stream)))


def device_error():
    code = ctypes.c_int(0)
    check(library().fs_device_error(ctypes.byref(code)))
    return code.value
