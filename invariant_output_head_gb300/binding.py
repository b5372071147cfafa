"""Thin ctypes binding of the C ABI in ``include/detlm_head.h``.

Argument marshalling only: every step of the output head runs in the CUDA
library. Functions keep the C names; ``Head`` wraps a handle for torch
tensors (device memory and streams come from PyTorch). There is no fallback:
if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib",
                         "libdetlm_head.so")

DETLM_BF16, DETLM_FP16, DETLM_INT8, DETLM_FP32, DETLM_E4M3 = 0, 1, 2, 3, 4
DTYPES = {"bf16": DETLM_BF16, "fp16": DETLM_FP16, "int8": DETLM_INT8, "e4m3": DETLM_E4M3}
DETLM_OK, DETLM_EINVAL, DETLM_EUNSUPPORTED, DETLM_ECUDA = 0, -1, -2, -3
DETLM_ETIMEOUT, DETLM_ENOMEM, DETLM_ETARGET = -4, -5, -6
DETLM_DEBUG_STALL = 1
DETLM_NO_TARGET = -1
DETLM_MAX_TOP = 32
DETLM_MAX_BEAMS, DETLM_MAX_BEAM_OUT = 32, 64

_vp, _i64, _i32, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
_SIGS = {
    "detlm_head_create": (_i32, [ctypes.POINTER(_vp), _vp, _i64, _i64, _i32]),
    "detlm_head_reserve": (_i32, [_vp, _i64]),
    "detlm_head_greedy": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _vp]),
    "detlm_head_logprob": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp]),
    "detlm_head_verify": (_i32, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "detlm_head_greedy_gated": (_i32, [_vp, _vp, _i64, ctypes.c_float, _vp, _vp, _vp, _vp, _vp,
                                       _vp]),
    "detlm_head_sample": (_i32, [_vp, _vp, _i64, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp]),
    "detlm_head_score": (_i32, [_vp, _vp, _vp, _i64, _i32, ctypes.c_float, _vp, _vp, _vp, _vp,
                                _vp, _vp]),
    "detlm_head_reserve_score": (_i32, [_vp, _i64, _i32]),
    "detlm_head_score_backward": (_i32, [_vp, _vp, _vp, _i64, ctypes.c_float, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _vp]),
    "detlm_head_reserve_backward": (_i32, [_vp, _i64]),
    "detlm_head_weights_changed": (_i32, [_vp, _vp]),
    "detlm_head_scaled_logits": (_i32, [_vp, _vp, _vp, _vp, _i64, _i32, _vp, _vp]),
    "detlm_quantize_blocks": (_i32, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp]),
    "detlm_head_block_scaled_logits": (_i32, [_vp, _vp, _vp, _vp, _i64, _i32, _vp, _vp]),
    "detlm_head_beam_select": (_i32, [_vp, _vp, _i32, _vp, _vp, ctypes.c_int32, _i64, _i32, _i32,
                                      ctypes.c_float, _vp, _vp, _vp, _vp]),
    "detlm_head_reserve_beams": (_i32, [_vp, _i64, _i32]),
    "detlm_beam_reorder": (_i32, [_vp, _i32, _vp, _i64, _i32, _i32, _i64, _vp]),
    "detlm_quantize_rows": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp]),
    "detlm_head_greedy_from_float": (_i32, [_vp, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "detlm_head_greedy_host": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _vp]),
    "detlm_head_logprob_host": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp]),
    "detlm_head_greedy_host_async": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _vp]),
    "detlm_head_logprob_host_async": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp]),
    "detlm_head_check": (_i32, [_vp, _vp]),
    "detlm_head_time_next": (_i32, [_vp, _vp, _vp]),
    "detlm_head_debug": (_i32, [_vp, _i32, _u64]),
    "detlm_head_tiles": (_i32, [_vp, _i64, ctypes.POINTER(ctypes.c_int32),
                                ctypes.POINTER(ctypes.c_int32)]),
    "detlm_head_destroy": (None, [_vp]),
    "detlm_status_string": (ctypes.c_char_p, [_i32]),
    "detlm_greedy_noalloc": (_i32, [_vp, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _vp]),
    "detlm_shard_range": (_i32, [_i64, _i32, _i32, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]),
    "detlm_head_create_shard": (_i32, [ctypes.POINTER(_vp), _vp, _i64, _i64, _i32, _i32, _i32]),
    "detlm_head_greedy_shard": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp]),
    "detlm_head_logprob_shard": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp]),
    "detlm_merge_greedy_shards": (_i32, [_vp, _i32, _i64, _i32, _vp, _vp, _vp]),
    "detlm_merge_logprob_shards": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp]),
}

_lib = None


@functools.lru_cache(None)
def _float_codes():
    import torch
    return {torch.bfloat16: DETLM_BF16, torch.float16: DETLM_FP16, torch.float32: DETLM_FP32}


def _float_dtype_code(x) -> int:
    code = _float_codes().get(x.dtype)
    if code is None:
        raise ValueError("float rows must be bfloat16, float16 or float32")
    return code


def _on_its_stream(call):
    """Run a call that was given a stream with that stream current: tensors
    that it makes are then the stream's (memory of the current stream's may
    still be in use by that stream's earlier work)."""
    at = call.__code__.co_varnames.index("stream")

    @functools.wraps(call)
    def run(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return call(*args, **kwargs)
        import torch
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)
    return run


def _on_device(t, call, *args, **kwargs):
    """call(...) with t's device current: a launch goes to the current one."""
    import torch
    if t.device.index == torch.cuda.current_device():
        return call(*args, **kwargs)
    with torch.cuda.device(t.device):
        return call(*args, **kwargs)


@_on_its_stream
def quantize_rows(x, stream=None):
    """Integer front end on a float CUDA tensor x [B, d]: returns (q int8
    [B, d], mult int32 [B], shift int32 [B])."""
    import torch
    xd = _float_dtype_code(x)
    if not x.is_cuda or not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous 2-D CUDA tensor")
    B, d = int(x.shape[0]), int(x.shape[1])
    q = torch.empty((B, d), dtype=torch.int8, device=x.device)
    mult = torch.empty(B, dtype=torch.int32, device=x.device)
    shift = torch.empty(B, dtype=torch.int32, device=x.device)
    detlm_quantize_rows(x.data_ptr(), xd, B, d, q.data_ptr(), mult.data_ptr(),
                        shift.data_ptr(), _stream_ptr(stream))
    return q, mult, shift


def block_buffers(B: int, d: int, block_rows: int = 1, device=None):
    """Output buffers (q, scale) for quantize_blocks of [B, d] rows."""
    import torch
    return (torch.empty((B, d), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((-(-B // block_rows), -(-d // 128)), dtype=torch.float32, device=device))


@_on_its_stream
def quantize_blocks(x, block_rows: int = 1, stream=None, out=None):
    """Float rows x [B, d] (bf16, fp16 or fp32 CUDA tensor, d a multiple of 16)
    in e4m3 with a power-of-two scale for each block of block_rows x 128
    elements (block_rows 1 for hidden rows, 128 for a weight). Returns (q
    float8_e4m3fn [B, d], scale float32 [ceil(B / block_rows), ceil(d / 128)])
    (detlm_quantize_blocks)."""
    import torch
    xd = _float_dtype_code(x)
    if not x.is_cuda or not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous 2-D CUDA tensor")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    B, d = x.shape
    if out is None:
        out = block_buffers(B, d, block_rows, x.device)
    q, scale = out
    if q.dtype != torch.float8_e4m3fn or q.shape != x.shape or not q.is_contiguous() \
            or q.device != x.device:
        raise ValueError("q must be a contiguous float8_e4m3fn tensor like x")
    if scale.dtype != torch.float32 or scale.shape != (-(-B // block_rows), -(-d // 128)) \
            or not scale.is_contiguous() or scale.device != x.device:
        raise ValueError("scale must be a contiguous float32 tensor, a value a block, on x's device")
    _on_device(x, lambda: detlm_quantize_blocks(x.data_ptr(), xd, B, d, block_rows, q.data_ptr(),
                                                scale.data_ptr(), _stream_ptr(stream)))
    return out


class DetlmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load the CUDA library (built by ``invariant_output_head_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -m invariant_output_head_gb300.build` (needs nvcc)")
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().detlm_status_string(status).decode()


def _check(st: int, what: str):
    if st != DETLM_OK:
        raise DetlmError(st, what)


# ---- the C entry points, by name (pointers and streams as ints) ----------

def detlm_head_create(W_ptr: int, V: int, d: int, dtype: int) -> int:
    out = _vp()
    _check(load_library().detlm_head_create(ctypes.byref(out), W_ptr, V, d, dtype),
           "detlm_head_create")
    return out.value


def detlm_head_reserve(handle: int, max_B: int) -> None:
    _check(load_library().detlm_head_reserve(handle, max_B), "detlm_head_reserve")


def detlm_head_greedy(handle, h_ptr, B, token_ptr, gap_ptr, logits_ptr, stream) -> None:
    _check(load_library().detlm_head_greedy(handle, h_ptr, B, token_ptr, gap_ptr,
                                            logits_ptr, stream), "detlm_head_greedy")


def detlm_head_logprob(handle, h_ptr, targets_ptr, B, logp_ptr, stream) -> None:
    _check(load_library().detlm_head_logprob(handle, h_ptr, targets_ptr, B, logp_ptr,
                                             stream), "detlm_head_logprob")


def detlm_head_greedy_gated(handle, h_ptr, B, tau, token_ptr, gap_ptr, logits_ptr,
                            base_token_ptr, margin_ptr, stream) -> None:
    _check(load_library().detlm_head_greedy_gated(handle, h_ptr, B, tau, token_ptr, gap_ptr,
                                                  logits_ptr, base_token_ptr, margin_ptr,
                                                  stream),
           "detlm_head_greedy_gated")


def detlm_head_sample(handle, h_ptr, B, temperature, seeds_ptr, positions_ptr, token_ptr,
                      score_gap_ptr, logits_ptr, stream) -> None:
    _check(load_library().detlm_head_sample(handle, h_ptr, B, temperature, seeds_ptr,
                                            positions_ptr, token_ptr, score_gap_ptr, logits_ptr,
                                            stream),
           "detlm_head_sample")


def detlm_head_score(handle, h_ptr, targets_ptr, B, top_k, temperature, logp_ptr, entropy_ptr,
                     lse_ptr, top_token_ptr, top_logp_ptr, stream) -> None:
    _check(load_library().detlm_head_score(handle, h_ptr, targets_ptr, B, top_k, temperature,
                                           logp_ptr, entropy_ptr, lse_ptr, top_token_ptr,
                                           top_logp_ptr, stream),
           "detlm_head_score")


def detlm_head_reserve_score(handle, max_B, top_k) -> None:
    _check(load_library().detlm_head_reserve_score(handle, max_B, top_k),
           "detlm_head_reserve_score")


def detlm_head_score_backward(handle, h_ptr, targets_ptr, B, temperature, lse_ptr, entropy_ptr,
                              dlogp_ptr, dentropy_ptr, dh_ptr, dW_ptr, stream) -> None:
    _check(load_library().detlm_head_score_backward(handle, h_ptr, targets_ptr, B, temperature,
                                                    lse_ptr, entropy_ptr, dlogp_ptr,
                                                    dentropy_ptr, dh_ptr, dW_ptr, stream),
           "detlm_head_score_backward")


def detlm_head_reserve_backward(handle, max_B) -> None:
    _check(load_library().detlm_head_reserve_backward(handle, max_B),
           "detlm_head_reserve_backward")


def detlm_head_weights_changed(handle, stream) -> None:
    _check(load_library().detlm_head_weights_changed(handle, stream),
           "detlm_head_weights_changed")


def detlm_head_scaled_logits(handle, q_ptr, x_scale_ptr, w_scale_ptr, B, out_dtype, out_ptr,
                             stream) -> None:
    _check(load_library().detlm_head_scaled_logits(handle, q_ptr, x_scale_ptr, w_scale_ptr, B,
                                                   out_dtype, out_ptr, stream),
           "detlm_head_scaled_logits")


def detlm_quantize_blocks(x_ptr, dtype, B, d, block_rows, q_ptr, scale_ptr, stream) -> None:
    _check(load_library().detlm_quantize_blocks(x_ptr, dtype, B, d, block_rows, q_ptr, scale_ptr,
                                                stream),
           "detlm_quantize_blocks")


def detlm_head_block_scaled_logits(handle, q_ptr, x_scale_ptr, w_scale_ptr, B, out_dtype, out_ptr,
                                   stream) -> None:
    _check(load_library().detlm_head_block_scaled_logits(handle, q_ptr, x_scale_ptr, w_scale_ptr,
                                                         B, out_dtype, out_ptr, stream),
           "detlm_head_block_scaled_logits")


def detlm_head_beam_select(handle, logits_ptr, logits_dtype, score_ptr, finished_ptr, end_token,
                           n_seq, beams, n_out, temperature, parent_ptr, token_ptr, out_score_ptr,
                           stream) -> None:
    _check(load_library().detlm_head_beam_select(handle, logits_ptr, logits_dtype, score_ptr,
                                                 finished_ptr, end_token, n_seq, beams, n_out,
                                                 temperature, parent_ptr, token_ptr,
                                                 out_score_ptr, stream),
           "detlm_head_beam_select")


def detlm_head_reserve_beams(handle, max_rows, n_out) -> None:
    _check(load_library().detlm_head_reserve_beams(handle, max_rows, n_out),
           "detlm_head_reserve_beams")


def detlm_beam_reorder(states_ptr, n_states, parent_ptr, n_seq, beams_in, beams_out, used,
                       stream) -> None:
    _check(load_library().detlm_beam_reorder(states_ptr, n_states, parent_ptr, n_seq, beams_in,
                                             beams_out, used, stream),
           "detlm_beam_reorder")


def detlm_quantize_rows(x_ptr, dtype, B, d, q_ptr, mult_ptr, shift_ptr, stream) -> None:
    _check(load_library().detlm_quantize_rows(x_ptr, dtype, B, d, q_ptr, mult_ptr, shift_ptr,
                                              stream),
           "detlm_quantize_rows")


def detlm_head_greedy_from_float(handle, x_ptr, x_dtype, B, token_ptr, gap_ptr, logits_ptr,
                                 mult_ptr, shift_ptr, stream) -> None:
    _check(load_library().detlm_head_greedy_from_float(handle, x_ptr, x_dtype, B, token_ptr,
                                                       gap_ptr, logits_ptr, mult_ptr, shift_ptr,
                                                       stream),
           "detlm_head_greedy_from_float")


def detlm_head_verify(handle, h_ptr, n_req, P, drafts_ptr, token_ptr, gap_ptr, logits_ptr,
                      accepted_ptr, stream) -> None:
    _check(load_library().detlm_head_verify(handle, h_ptr, n_req, P, drafts_ptr, token_ptr,
                                            gap_ptr, logits_ptr, accepted_ptr, stream),
           "detlm_head_verify")


def detlm_head_greedy_host(handle, h_ptr, B, token_ptr, gap_ptr, logits_ptr, stream) -> None:
    _check(load_library().detlm_head_greedy_host(handle, h_ptr, B, token_ptr, gap_ptr,
                                                 logits_ptr, stream),
           "detlm_head_greedy_host")


def detlm_head_logprob_host(handle, h_ptr, targets_ptr, B, logp_ptr, stream) -> None:
    _check(load_library().detlm_head_logprob_host(handle, h_ptr, targets_ptr, B,
                                                  logp_ptr, stream),
           "detlm_head_logprob_host")


def detlm_head_greedy_host_async(handle, h_ptr, B, token_ptr, gap_ptr, logits_ptr,
                                 stream) -> None:
    _check(load_library().detlm_head_greedy_host_async(handle, h_ptr, B, token_ptr, gap_ptr,
                                                       logits_ptr, stream),
           "detlm_head_greedy_host_async")


def detlm_head_logprob_host_async(handle, h_ptr, targets_ptr, B, logp_ptr, stream) -> None:
    _check(load_library().detlm_head_logprob_host_async(handle, h_ptr, targets_ptr, B,
                                                        logp_ptr, stream),
           "detlm_head_logprob_host_async")


def detlm_head_check(handle, stream) -> int:
    return load_library().detlm_head_check(handle, stream)


def detlm_head_time_next(handle, start_evt: int, stop_evt: int) -> None:
    _check(load_library().detlm_head_time_next(handle, start_evt, stop_evt),
           "detlm_head_time_next")


def detlm_head_debug(handle, flags: int, timeout_ns: int = 0) -> None:
    _check(load_library().detlm_head_debug(handle, flags, timeout_ns), "detlm_head_debug")


def detlm_head_tiles(handle, B: int):
    nv, nc = ctypes.c_int32(), ctypes.c_int32()
    _check(load_library().detlm_head_tiles(handle, B, ctypes.byref(nv), ctypes.byref(nc)),
           "detlm_head_tiles")
    return nv.value, nc.value


def detlm_head_destroy(handle) -> None:
    if handle:
        load_library().detlm_head_destroy(handle)


def detlm_status_string(status: int) -> str:
    return status_string(status)


def detlm_greedy_noalloc(W_ptr, V, d, dtype, h_ptr, B, token_ptr, gap_ptr, logits_ptr,
                         err_ptr, stream) -> None:
    """Greedy call that allocates no device memory (its workspace is a static
    device array inside the library); for callers that may not allocate."""
    _check(load_library().detlm_greedy_noalloc(W_ptr, V, d, dtype, h_ptr, B, token_ptr,
                                               gap_ptr, logits_ptr, err_ptr, stream),
           "detlm_greedy_noalloc")


def detlm_shard_range(V: int, P: int, rank: int):
    """(v_begin, v_end): the vocabulary rows shard `rank` of P holds (host only)."""
    a, b = _i64(), _i64()
    _check(load_library().detlm_shard_range(V, P, rank, ctypes.byref(a), ctypes.byref(b)),
           "detlm_shard_range")
    return a.value, b.value


def detlm_head_create_shard(W_ptr: int, V: int, d: int, dtype: int, P: int, rank: int) -> int:
    out = _vp()
    _check(load_library().detlm_head_create_shard(ctypes.byref(out), W_ptr, V, d, dtype, P, rank),
           "detlm_head_create_shard")
    return out.value


def detlm_head_greedy_shard(handle, h_ptr, B, rec_ptr, logits_ptr, stream) -> None:
    _check(load_library().detlm_head_greedy_shard(handle, h_ptr, B, rec_ptr, logits_ptr, stream),
           "detlm_head_greedy_shard")


def detlm_head_logprob_shard(handle, h_ptr, targets_ptr, B, rec_ptr, stream) -> None:
    _check(load_library().detlm_head_logprob_shard(handle, h_ptr, targets_ptr, B, rec_ptr,
                                                   stream),
           "detlm_head_logprob_shard")


def detlm_merge_greedy_shards(recs_ptr, P, B, dtype, token_ptr, gap_ptr, stream) -> None:
    _check(load_library().detlm_merge_greedy_shards(recs_ptr, P, B, dtype, token_ptr, gap_ptr,
                                                    stream),
           "detlm_merge_greedy_shards")


def detlm_merge_logprob_shards(recs_ptr, P, B, V, targets_ptr, logp_ptr, err_ptr, stream) -> None:
    _check(load_library().detlm_merge_logprob_shards(recs_ptr, P, B, V, targets_ptr, logp_ptr,
                                                     err_ptr, stream),
           "detlm_merge_logprob_shards")


# ---- torch convenience wrapper ------------------------------------------

def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_ptr(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    import torch
    # (torch.cuda.current_stream() makes an object, which takes longer than a launch)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


class Score(NamedTuple):
    """What Head.score returns (and the buffers it can be given as `out`)."""
    logp: object        # float32 [B] (None without targets)
    entropy: object     # float32 [B]
    lse: object         # float32 [B]
    top_token: object   # int32 [B, top_k] (None when top_k is 0)
    top_logp: object    # float32 [B, top_k]


class Beams(NamedTuple):
    """What Head.beam_select returns (and the buffers it can be given as `out`)."""
    parent: object      # int32 [n_seq, n_out]: the beam continued, -1 for none
    token: object       # int32 [n_seq, n_out]
    score: object       # float32 [n_seq, n_out]


def beam_buffers(n_seq: int, n_out: int, device=None) -> Beams:
    """Output buffers for Head.beam_select (pass them as `out`)."""
    import torch
    i32 = dict(dtype=torch.int32, device=device)
    return Beams(torch.empty((n_seq, n_out), **i32), torch.empty((n_seq, n_out), **i32),
                 torch.empty((n_seq, n_out), dtype=torch.float32, device=device))


def _matrix(t, name, shape, dtype, device):
    """A contiguous CUDA tensor of the shape and type, or a ValueError."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {device}")


def _vector(t, name, B, dtype, device):
    """A contiguous 1-D CUDA tensor of B values, or a ValueError."""
    if t.dtype != dtype or not t.is_cuda or t.dim() != 1 or t.shape[0] != B \
            or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor [{B}]")


class Head:
    """One output head over a device weight W [V, d] (bf16, fp16, int8 or
    float8_e4m3fn tensor; the last has block_scaled_logits and beam_select only).

    The handle borrows W: keep the tensor alive while the Head is in use.
    """

    def __init__(self, W, dtype: str | None = None):
        import torch
        if dtype is None:
            dtype = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.int8: "int8",
                     torch.float8_e4m3fn: "e4m3"}[W.dtype]
        if not W.is_cuda or not W.is_contiguous() or W.dim() != 2:
            raise ValueError("W must be a contiguous 2-D CUDA tensor [V, d]")
        self.W = W
        self.dtype = dtype
        self.V, self.d = int(W.shape[0]), int(W.shape[1])
        self.handle = detlm_head_create(W.data_ptr(), self.V, self.d, DTYPES[dtype])

    def close(self):
        if getattr(self, "handle", None):
            detlm_head_destroy(self.handle)
            self.handle = None

    def reserve(self, max_B: int) -> None:
        """Workspace (and, for an int8 head, the wide path's fp16 copies) for
        calls of up to max_B rows: such calls then allocate nothing and can be
        captured into a CUDA graph (detlm_head_reserve)."""
        detlm_head_reserve(self.handle, int(max_B))

    def __del__(self):
        try:
            self.close()
        except Exception:   # noqa: BLE001 - interpreter shutdown
            pass

    def _check_h(self, h):
        if not h.is_cuda or not h.is_contiguous() or h.dim() != 2 or h.shape[1] != self.d:
            raise ValueError(f"h must be a contiguous CUDA tensor [B, {self.d}]")
        # the library takes a bare pointer: rows of another type would be
        # misread, of a smaller one past their end
        if h.dtype != self.W.dtype:
            raise ValueError(f"h must have the head's dtype, {self.W.dtype}")
        if h.device != self.W.device:
            raise ValueError(f"h must be on the head's device, {self.W.device}")

    @_on_its_stream
    def greedy(self, h, with_logits: bool = False, stream=None, out=None):
        """Returns (token int32 [B], gap [B], logits [B, V] or None) on h's device."""
        import torch
        self._check_h(h)
        B = int(h.shape[0])
        gdt = torch.int32 if self.dtype == "int8" else torch.float32
        if out is None:
            token = torch.empty(B, dtype=torch.int32, device=h.device)
            gap = torch.empty(B, dtype=gdt, device=h.device)
            logits = torch.empty((B, self.V), dtype=gdt, device=h.device) if with_logits else None
        else:
            token, gap, logits = out
        detlm_head_greedy(self.handle, h.data_ptr(), B, token.data_ptr(), gap.data_ptr(),
                          logits.data_ptr() if logits is not None else None,
                          _stream_ptr(stream))
        return token, gap, logits

    @_on_its_stream
    def logprob(self, h, targets, stream=None, out=None):
        import torch
        self._check_h(h)
        B = int(h.shape[0])
        if targets.dtype != torch.int32 or not targets.is_cuda or targets.numel() != B:
            raise ValueError("targets must be an int32 CUDA tensor [B]")
        logp = torch.empty(B, dtype=torch.float32, device=h.device) if out is None else out
        detlm_head_logprob(self.handle, h.data_ptr(), targets.data_ptr(), B, logp.data_ptr(),
                           _stream_ptr(stream))
        return logp

    def score_buffers(self, B: int, top_k: int = 0, targets: bool = True) -> Score:
        """Output buffers for score calls of B rows (pass them as `out`)."""
        import torch
        f32 = dict(dtype=torch.float32, device=self.W.device)
        top = (torch.empty((B, top_k), dtype=torch.int32, device=self.W.device) if top_k else None)
        return Score(torch.empty(B, **f32) if targets else None, torch.empty(B, **f32),
                     torch.empty(B, **f32), top, torch.empty((B, top_k), **f32) if top_k else None)

    @_on_its_stream
    def score(self, h, targets=None, top_k: int = 0, temperature: float = 1.0, stream=None,
              out: Score | None = None) -> Score:
        """Log-probability of targets int32 [B] (DETLM_NO_TARGET: nothing to
        score, 0), entropy and log-sum-exp of each row's distribution at the
        given temperature, and its top_k most likely tokens with their
        log-probabilities (detlm_head_score)."""
        import torch
        self._check_h(h)
        B = int(h.shape[0])
        if targets is not None:
            _vector(targets, "targets", B, torch.int32, h.device)
        if out is None:
            out = self.score_buffers(B, top_k, targets is not None)
        else:
            for name, t in (("out.logp", out.logp), ("out.entropy", out.entropy),
                            ("out.lse", out.lse)):
                if t is not None:
                    _vector(t, name, B, torch.float32, h.device)
            if (out.logp is None) != (targets is None):
                raise ValueError("out.logp goes with targets")
            if top_k:
                for t, dt in ((out.top_token, torch.int32), (out.top_logp, torch.float32)):
                    if t is None or t.dtype != dt or tuple(t.shape) != (B, top_k) \
                            or not t.is_contiguous() or t.device != h.device:
                        raise ValueError("out.top_token and out.top_logp must be contiguous "
                                         f"[{B}, {top_k}] tensors")
        ptr = _ptr
        detlm_head_score(self.handle, h.data_ptr(), ptr(targets), B, top_k, temperature,
                         ptr(out.logp), ptr(out.entropy), ptr(out.lse),
                         ptr(out.top_token) if top_k else None,
                         ptr(out.top_logp) if top_k else None, _stream_ptr(stream))
        return out

    def reserve_score(self, max_B: int, top_k: int = 0) -> None:
        """Workspace for score calls of up to max_B rows and top_k alternatives."""
        detlm_head_reserve_score(self.handle, int(max_B), int(top_k))

    @_on_its_stream
    def score_backward(self, h, targets, lse, entropy, dlogp, dentropy=None,
                       temperature: float = 1.0, need_dh: bool = True, need_dW: bool = True,
                       stream=None, out=None):
        """Gradients (dh [B, d], dW [V, d]) in the head's type of a loss whose
        gradients with respect to score's logp and entropy are dlogp and
        dentropy, float32 [B] (detlm_head_score_backward). lse and entropy are
        what score returned. One that is not needed is None."""
        import torch
        self._check_h(h)
        B = int(h.shape[0])
        _vector(targets, "targets", B, torch.int32, h.device)
        for name, t in (("lse", lse), ("dlogp", dlogp), ("dentropy", dentropy),
                        ("entropy", entropy if dentropy is not None else None)):
            if t is not None:
                _vector(t, name, B, torch.float32, h.device)
        if out is None:
            dh = torch.empty_like(h) if need_dh else None
            dW = torch.empty_like(self.W) if need_dW else None
        else:
            dh, dW = out
            for name, t, like in (("dh", dh, h), ("dW", dW, self.W)):
                if t is not None and (t.dtype != like.dtype or t.shape != like.shape
                                      or not t.is_contiguous() or t.device != like.device):
                    raise ValueError(f"{name} must be like {'h' if name == 'dh' else 'W'}")
        detlm_head_score_backward(self.handle, h.data_ptr(), targets.data_ptr(), B, temperature,
                                  lse.data_ptr(),
                                  entropy.data_ptr() if dentropy is not None else None,
                                  dlogp.data_ptr(), _ptr(dentropy), _ptr(dh), _ptr(dW),
                                  _stream_ptr(stream))
        return dh, dW

    def reserve_backward(self, max_B: int) -> None:
        """Workspace for gradient calls of up to max_B rows."""
        detlm_head_reserve_backward(self.handle, int(max_B))

    def weights_changed(self, stream=None) -> None:
        """Tell the head that W was changed in place on the stream; graphs
        captured before the change use the new W from then on
        (detlm_head_weights_changed)."""
        detlm_head_weights_changed(self.handle, _stream_ptr(stream))

    @_on_its_stream
    def scaled_logits(self, q, x_scale, w_scale, out_dtype=None, stream=None, out=None):
        """int8 head: (q . W^T) * x_scale[:, None] * w_scale[None, :] as
        float32 (default), bfloat16 or float16 [B, V]; q int8 [B, d], x_scale
        float32 [B] (one scale a token), w_scale float32 [V] (one a channel)."""
        import torch
        if self.dtype != "int8":
            raise DetlmError(DETLM_EUNSUPPORTED, "scaled_logits")
        self._check_h(q)
        B = int(q.shape[0])
        _vector(x_scale, "x_scale", B, torch.float32, q.device)
        _vector(w_scale, "w_scale", self.V, torch.float32, q.device)
        if out is None:
            out = torch.empty((B, self.V), dtype=out_dtype or torch.float32, device=q.device)
        elif (out.shape != (B, self.V) or not out.is_contiguous() or out.device != q.device
              or (out_dtype is not None and out.dtype != out_dtype)):
            raise ValueError(f"out must be a contiguous [{B}, {self.V}] CUDA tensor")
        detlm_head_scaled_logits(self.handle, q.data_ptr(), x_scale.data_ptr(),
                                 w_scale.data_ptr(), B, _float_dtype_code(out), out.data_ptr(),
                                 _stream_ptr(stream))
        return out

    @_on_its_stream
    def block_scaled_logits(self, q, x_scale, w_scale, out_dtype=None, stream=None, out=None):
        """e4m3 head: the logits [B, V] of rows q float8_e4m3fn [B, d] as
        float32 (default), bfloat16 or float16, with x_scale float32 [B, ceil(d
        / 128)] for each row's blocks and w_scale float32 [ceil(V / 128), ceil(d
        / 128)] for W's (detlm_head_block_scaled_logits)."""
        import torch
        if self.dtype != "e4m3":
            raise DetlmError(DETLM_EUNSUPPORTED, "block_scaled_logits")
        self._check_h(q)
        B, blocks = q.shape[0], -(-self.d // 128)
        _matrix(x_scale, "x_scale", (B, blocks), torch.float32, q.device)
        _matrix(w_scale, "w_scale", (-(-self.V // 128), blocks), torch.float32, q.device)
        if out is None:
            out = torch.empty((B, self.V), dtype=out_dtype or torch.float32, device=q.device)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out has another dtype")
        _matrix(out, "out", (B, self.V), out.dtype, q.device)
        code = _float_dtype_code(out)
        _on_device(q, lambda: detlm_head_block_scaled_logits(
            self.handle, q.data_ptr(), x_scale.data_ptr(), w_scale.data_ptr(), B, code,
            out.data_ptr(), _stream_ptr(stream)))
        return out

    @_on_its_stream
    def beam_select(self, logits, scores, n_out: int, temperature: float = 1.0, finished=None,
                    end_token: int = 0, stream=None, out: Beams | None = None) -> Beams:
        """The n_out best continuations of each sequence's beams: logits
        [n_seq * beams, V] (float32, bfloat16 or float16) of this head, scores
        float32 [n_seq, beams] the beams' log-probabilities so far. Beams marked
        in finished (bool or uint8 [n_seq, beams]) stay as they are, with
        end_token (detlm_head_beam_select). out.score may be scores."""
        import torch
        if scores.dim() != 2:
            raise ValueError("scores must be [n_seq, beams]")
        n_seq, beams = scores.shape
        device = self.W.device
        _matrix(scores, "scores", (n_seq, beams), torch.float32, device)
        _matrix(logits, "logits", (n_seq * beams, self.V), logits.dtype, device)
        code = _float_dtype_code(logits)
        if finished is not None:
            if finished.dtype not in (torch.bool, torch.uint8):
                raise ValueError("finished must be a bool or uint8 tensor")
            _matrix(finished, "finished", (n_seq, beams), finished.dtype, device)
            # (C integers would take the low bits of larger numbers, here and below)
            if not 0 <= end_token < self.V:
                raise DetlmError(DETLM_EINVAL, "beam_select: end_token")
        if not 1 <= n_out <= DETLM_MAX_BEAM_OUT:
            raise DetlmError(DETLM_EINVAL, "beam_select: n_out")
        if out is None:
            out = beam_buffers(n_seq, n_out, device)
        else:
            _matrix(out.parent, "out.parent", (n_seq, n_out), torch.int32, device)
            _matrix(out.token, "out.token", (n_seq, n_out), torch.int32, device)
            _matrix(out.score, "out.score", (n_seq, n_out), torch.float32, device)
            gap = out.score.data_ptr() - scores.data_ptr()
            if -4 * out.score.numel() < gap < 4 * scores.numel() and (gap or n_out != beams):
                raise ValueError("out.score must be scores, or apart from it")
        _on_device(scores, lambda: detlm_head_beam_select(
            self.handle, logits.data_ptr(), code, scores.data_ptr(), _ptr(finished), end_token,
            n_seq, beams, n_out, temperature, out.parent.data_ptr(), out.token.data_ptr(),
            out.score.data_ptr(), _stream_ptr(stream)))
        return out

    def reserve_beams(self, max_rows: int, n_out: int) -> None:
        """Workspace for selections of up to max_rows = n_seq * beams rows and
        n_out continuations."""
        if not 0 <= max_rows < 1 << 31 or not 1 <= n_out <= DETLM_MAX_BEAM_OUT:
            raise DetlmError(DETLM_EINVAL, "reserve_beams")
        _on_device(self.W, lambda: detlm_head_reserve_beams(self.handle, int(max_rows), int(n_out)))

    @_on_its_stream
    def greedy_gated(self, h, tau: float = 0.001, with_logits: bool = False, stream=None):
        """Margin-gated greedy call. Returns (token, gap, logits or None,
        base_token, margin)."""
        import torch
        self._check_h(h)
        B = int(h.shape[0])
        token = torch.empty(B, dtype=torch.int32, device=h.device)
        gap = torch.empty(B, dtype=torch.float32, device=h.device)
        base = torch.empty(B, dtype=torch.int32, device=h.device)
        margin = torch.empty(B, dtype=torch.float32, device=h.device)
        logits = (torch.empty((B, self.V), dtype=torch.float32, device=h.device)
                  if with_logits else None)
        detlm_head_greedy_gated(self.handle, h.data_ptr(), B, float(tau), token.data_ptr(),
                                gap.data_ptr(), logits.data_ptr() if logits is not None else None,
                                base.data_ptr(), margin.data_ptr(), _stream_ptr(stream))
        return token, gap, logits, base, margin

    @_on_its_stream
    def sample(self, h, temperature, seeds, positions, with_logits: bool = False, stream=None):
        """Seeded sampling. seeds, positions: int64/uint64 CUDA tensors [B]
        (read as unsigned 64-bit). Returns (token, score_gap, logits or None)."""
        import torch
        self._check_h(h)
        B = int(h.shape[0])
        for name, t in (("seeds", seeds), ("positions", positions)):
            if (not t.is_cuda or t.dim() != 1 or int(t.shape[0]) != B
                    or t.element_size() != 8 or t.is_floating_point()):
                raise ValueError(f"{name} must be a 64-bit integer CUDA tensor [B]")
        token = torch.empty(B, dtype=torch.int32, device=h.device)
        gap = torch.empty(B, dtype=torch.float32, device=h.device)
        logits = (torch.empty((B, self.V), dtype=torch.float32, device=h.device)
                  if with_logits else None)
        detlm_head_sample(self.handle, h.data_ptr(), B, float(temperature),
                          seeds.contiguous().data_ptr(), positions.contiguous().data_ptr(),
                          token.data_ptr(), gap.data_ptr(),
                          logits.data_ptr() if logits is not None else None, _stream_ptr(stream))
        return token, gap, logits

    @_on_its_stream
    def greedy_from_float(self, x, with_logits: bool = False, stream=None):
        """int8 head fed by float rows x [B, d] (bf16, fp16 or fp32 CUDA
        tensor). Returns (token, gap, logits or None, mult, shift)."""
        import torch
        if self.dtype != "int8":
            raise DetlmError(DETLM_EUNSUPPORTED, "greedy_from_float")
        xd = _float_dtype_code(x)
        if not x.is_cuda or not x.is_contiguous() or x.dim() != 2 or x.shape[1] != self.d:
            raise ValueError(f"x must be a contiguous CUDA tensor [B, {self.d}]")
        B = int(x.shape[0])
        token = torch.empty(B, dtype=torch.int32, device=x.device)
        gap = torch.empty(B, dtype=torch.int32, device=x.device)
        mult = torch.empty(B, dtype=torch.int32, device=x.device)
        shift = torch.empty(B, dtype=torch.int32, device=x.device)
        logits = (torch.empty((B, self.V), dtype=torch.int32, device=x.device)
                  if with_logits else None)
        detlm_head_greedy_from_float(self.handle, x.data_ptr(), xd, B, token.data_ptr(),
                                     gap.data_ptr(),
                                     logits.data_ptr() if logits is not None else None,
                                     mult.data_ptr(), shift.data_ptr(), _stream_ptr(stream))
        return token, gap, logits, mult, shift

    @_on_its_stream
    def verify(self, h, drafts, with_logits: bool = False, stream=None):
        """Greedy speculative verify. h [R*P, d] request-major, drafts int32
        [R, P]. Returns (token [R*P], gap, logits or None, accepted [R])."""
        import torch
        self._check_h(h)
        if drafts.dtype != torch.int32 or not drafts.is_cuda or drafts.dim() != 2:
            raise ValueError("drafts must be an int32 CUDA tensor [R, P]")
        R, P = int(drafts.shape[0]), int(drafts.shape[1])
        if R * P != int(h.shape[0]):
            raise ValueError("h must hold R * P rows")
        gdt = torch.int32 if self.dtype == "int8" else torch.float32
        token = torch.empty(R * P, dtype=torch.int32, device=h.device)
        gap = torch.empty(R * P, dtype=gdt, device=h.device)
        logits = torch.empty((R * P, self.V), dtype=gdt, device=h.device) if with_logits else None
        accepted = torch.empty(R, dtype=torch.int32, device=h.device)
        detlm_head_verify(self.handle, h.data_ptr(), R, P, drafts.contiguous().data_ptr(),
                          token.data_ptr(), gap.data_ptr(),
                          logits.data_ptr() if logits is not None else None,
                          accepted.data_ptr(), _stream_ptr(stream))
        return token, gap, logits, accepted

    def check(self, stream=None) -> int:
        return detlm_head_check(self.handle, _stream_ptr(stream))

    def tiles(self, B: int):
        return detlm_head_tiles(self.handle, B)


# ---- the beams' states ----------------------------------------------------

class _State(ctypes.Structure):       # detlm_beam_state_t
    _fields_ = [("src", _vp), ("dst", _vp), ("src_row", _i64), ("dst_row", _i64),
                ("src_seg", _i64), ("dst_seg", _i64), ("n_seg", _i64), ("seg_bytes", _i64),
                ("position_bytes", _i64)]


def _pieces(t, axis):
    """Layout of a row of t, [rows, ...], in bytes: (row stride, piece stride,
    pieces, bytes a position, positions). A row is equal contiguous pieces, each
    of the positions along `axis` (a piece is one position without it)."""
    size = t.element_size()
    dims = [(n, s * size) for n, s in zip(t.shape, t.stride())]
    axis = len(dims) if axis is None else axis

    def fold(part):
        """The axes as one of equal steps: (count, step), the step None for one."""
        count, step = 1, None
        for n, s in reversed(part):
            if n == 1:
                continue
            if step is None:
                step = s
            elif s != step * count:
                raise ValueError("the rows of a state must be equal contiguous pieces")
            count *= n
        return count, step

    if axis == len(dims):
        # contiguous axes at the end make the piece
        k, each = len(dims), size
        while k > 1 and (dims[k - 1][0] == 1 or dims[k - 1][1] == each):
            each *= dims[k - 1][0]
            k -= 1
        positions = 1
    else:
        k = axis
        n, step = fold(dims[axis + 1:])
        each = n * size
        if step is not None and step != size:
            raise ValueError("the rows of a state must be equal contiguous pieces")
        positions, s = dims[axis]
        if positions > 1 and s != each:
            raise ValueError("the positions of a state must be contiguous")
    n_seg, step = fold(dims[1:k])
    return dims[0][1], step or 0, n_seg, each, positions


def _shared(a, b=None):
    """Whether two states' rows (address, row step, rows, piece step, pieces,
    bytes of a piece) share a byte; of one state: whether two of its pieces do.
    Exact for states of one layout and for rows that lie apart; other states
    whose memory interleaves count as sharing it."""
    own, b = b is None, a if b is None else b
    extent = [(n - 1) * seg + size for _, _, _, seg, n, size in (a, b)]   # of a row
    at = b[0] - a[0]
    if not own and (at >= (a[2] - 1) * a[1] + extent[0] or -at >= (b[2] - 1) * b[1] + extent[1]):
        return False
    step, seg, size = a[1], a[3], a[5]
    if b[1] != step and a[2] > 1 and b[2] > 1:
        return True
    if b[2] > 1:
        step = b[1]
    if a[2] == b[2] == 1:
        step = sum(extent)                       # (any)
    if step == 0:
        return True
    # rows of b that lie `first` to `last` rows from one of a and reach into it
    first = max(1 - a[2], -((at + extent[1] - 1) // step))
    last = min(b[2] - 1, (extent[0] - 1 - at) // step)
    for d in range(first, last + 1):
        off = at + d * step
        if b[3:] != a[3:]:
            return True
        if a[4] == 1:
            if not (own and d == 0):
                return True
            continue
        # pieces of b that lie k pieces from one of a
        near = -off // seg if seg else 0
        for k in (near, near + 1):
            k = max(1 - a[4], min(a[4] - 1, k))
            if abs(off + k * seg) < size and not (own and d == 0 and k == 0):
                return True
        if own and d == 0 and seg < size:
            return True
    return False


class BeamStates:
    """The tensors that hold the states of beams (caches, token histories),
    rows [n_seq * beams, ...] first, and their reordering (detlm_beam_reorder).

    Rows move in place, or, with `out`, into other tensors of the same types
    and shapes (but for the number of rows, where a step changes the number of
    beams). token_dim names the axis of positions of each state (one number, or
    one a state, None for a state without), of which reorder(used=n) moves the
    first n. A row has to be equal contiguous pieces (any one axis, or several
    that make one, strided), and no two states share memory, nor out any with the
    states. The tensors are kept; their addresses and strides are read once, here.
    """

    def __init__(self, states, out=None, token_dim=None):
        states = list(states)
        outs = states if out is None else list(out)
        dims = list(token_dim) if isinstance(token_dim, (list, tuple)) else [token_dim] * len(states)
        if not states or len(outs) != len(states) or len(dims) != len(states):
            raise ValueError("states, out and token_dim must be as many, and at least one")
        self.states, self.out = states, outs
        self.device = states[0].device
        self.rows_in, self.rows_out = int(states[0].shape[0]), int(outs[0].shape[0])
        self._table = (_State * len(states))()
        self._address = ctypes.addressof(self._table)
        self.positions = None
        for e, s, o, dim in zip(self._table, states, outs, dims):
            for t, rows in ((s, self.rows_in), (o, self.rows_out)):
                if not t.is_cuda or t.device != self.device or t.dim() < 1 or t.shape[0] != rows:
                    raise ValueError("states must be CUDA tensors of one device and as many rows")
            if s.dtype != o.dtype or s.shape[1:] != o.shape[1:]:
                raise ValueError("out must be like the states")
            if dim is not None:
                dim = dim + s.dim() if dim < 0 else dim
                if not 1 <= dim < s.dim():
                    raise ValueError("token_dim must be an axis behind the rows")
            a, b = _pieces(s, dim), _pieces(o, dim)
            if a[2:] != b[2:]:
                raise ValueError("a state and its out must have rows of the same pieces")
            e.src, e.dst = s.data_ptr(), o.data_ptr()
            e.src_row, e.src_seg = a[:2]
            e.dst_row, e.dst_seg = b[:2]
            e.n_seg, each, positions = a[2:]
            e.seg_bytes = each * positions
            if s.numel() == 0:
                e.n_seg = 0
            e.position_bytes = each if dim is not None else 0
            if dim is not None:
                self.positions = positions if self.positions is None else min(positions, self.positions)
        self._check_overlap(out is None)

    def _check_overlap(self, in_place):
        rows = [(e.dst, e.dst_row, self.rows_out, e.dst_seg, e.n_seg, e.seg_bytes)
                for e in self._table if e.n_seg and self.rows_out]
        for i, a in enumerate(rows):
            if _shared(a):
                raise ValueError("an output has more than one element at one place")
            for b in rows[:i]:
                if _shared(a, b):
                    raise ValueError("two states share memory")
        if in_place:
            return
        for a in rows:
            for e in self._table:
                if e.n_seg and _shared(a, (e.src, e.src_row, self.rows_in, e.src_seg, e.n_seg,
                                           e.seg_bytes)):
                    raise ValueError("out overlaps a state")

    def reorder(self, parent, used: int | None = None, stream=None) -> None:
        """Row s * beams + j becomes row s * beams + parent[s, j] (int32 [n_seq,
        beams], as beam_select returns them; one outside the sequence's beams
        leaves its row as it was). used: positions that hold something (all by
        default)."""
        import torch
        if parent.dtype != torch.int32 or parent.dim() != 2 or not parent.is_contiguous() \
                or parent.device != self.device:
            raise ValueError(f"parent must be a contiguous int32 tensor [n_seq, beams] on {self.device}")
        n_seq, beams = parent.shape
        if n_seq * beams != self.rows_out or (n_seq and self.rows_in % n_seq):
            raise ValueError(f"parent must have {self.rows_out} entries, for {self.rows_in} rows")
        if n_seq == 0:
            return
        if used is not None and (self.positions is None or not 0 <= used <= self.positions):
            raise ValueError("used must be a number of the states' positions")
        _on_device(parent, lambda: detlm_beam_reorder(
            self._address, len(self._table), parent.data_ptr(), n_seq, self.rows_in // n_seq,
            beams, -1 if used is None else used, _stream_ptr(stream)))


# ---- vocabulary-parallel heads -------------------------------------------

SHARD_REC_INT32S = 4     # one detlm_shard_rec_t = 16 bytes = 4 int32 words


class ShardHead(Head):
    """Shard `rank` of P of a head split by vocabulary rows. W_shard holds the
    rows detlm_shard_range(V, P, rank) of the full weight (V rows in all)."""

    def __init__(self, W_shard, V: int, P: int, rank: int, dtype: str | None = None):
        import torch
        if dtype is None:
            dtype = {torch.bfloat16: "bf16", torch.float16: "fp16",
                     torch.int8: "int8"}[W_shard.dtype]
        if not W_shard.is_cuda or not W_shard.is_contiguous() or W_shard.dim() != 2:
            raise ValueError("W_shard must be a contiguous 2-D CUDA tensor")
        v0, v1 = detlm_shard_range(V, P, rank)
        if int(W_shard.shape[0]) != v1 - v0:
            raise ValueError(f"shard {rank} of {P} holds rows [{v0}, {v1})")
        self.W = W_shard
        self.dtype = dtype
        self.V, self.d = int(W_shard.shape[0]), int(W_shard.shape[1])
        self.V_total, self.P, self.rank, self.v_begin, self.v_end = V, P, rank, v0, v1
        self.handle = detlm_head_create_shard(W_shard.data_ptr(), V, self.d, DTYPES[dtype], P, rank)

    @_on_its_stream
    def greedy_records(self, h, with_logits: bool = False, stream=None):
        """Records int32 [B, 4] (detlm_shard_rec_t) and the shard's logits or None."""
        import torch
        self._check_h(h)
        B = int(h.shape[0])
        rec = torch.empty((B, SHARD_REC_INT32S), dtype=torch.int32, device=h.device)
        gdt = torch.int32 if self.dtype == "int8" else torch.float32
        logits = torch.empty((B, self.V), dtype=gdt, device=h.device) if with_logits else None
        detlm_head_greedy_shard(self.handle, h.data_ptr(), B, rec.data_ptr(),
                                logits.data_ptr() if logits is not None else None,
                                _stream_ptr(stream))
        return rec, logits

    @_on_its_stream
    def logprob_records(self, h, targets, stream=None):
        import torch
        self._check_h(h)
        B = int(h.shape[0])
        if targets.dtype != torch.int32 or not targets.is_cuda or targets.numel() != B:
            raise ValueError("targets must be an int32 CUDA tensor [B]")
        rec = torch.empty((B, SHARD_REC_INT32S), dtype=torch.int32, device=h.device)
        detlm_head_logprob_shard(self.handle, h.data_ptr(), targets.data_ptr(), B, rec.data_ptr(),
                                 _stream_ptr(stream))
        return rec


@_on_its_stream
def merge_greedy(recs, dtype: str, stream=None):
    """recs int32 [P, B, 4] (shard-major) -> (token int32 [B], gap [B])."""
    import torch
    if recs.dtype != torch.int32 or recs.dim() != 3 or recs.shape[2] != SHARD_REC_INT32S:
        raise ValueError("recs must be an int32 tensor [P, B, 4]")
    recs = recs.contiguous()
    P, B = int(recs.shape[0]), int(recs.shape[1])
    token = torch.empty(B, dtype=torch.int32, device=recs.device)
    gap = torch.empty(B, dtype=torch.int32 if dtype == "int8" else torch.float32,
                      device=recs.device)
    detlm_merge_greedy_shards(recs.data_ptr(), P, B, DTYPES[dtype], token.data_ptr(),
                              gap.data_ptr(), _stream_ptr(stream))
    return token, gap


@_on_its_stream
def merge_logprob(recs, V: int, targets, err=None, stream=None):
    """recs int32 [P, B, 4] -> logp float32 [B]."""
    import torch
    if recs.dtype != torch.int32 or recs.dim() != 3 or recs.shape[2] != SHARD_REC_INT32S:
        raise ValueError("recs must be an int32 tensor [P, B, 4]")
    recs = recs.contiguous()
    P, B = int(recs.shape[0]), int(recs.shape[1])
    logp = torch.empty(B, dtype=torch.float32, device=recs.device)
    detlm_merge_logprob_shards(recs.data_ptr(), P, B, V, targets.data_ptr(), logp.data_ptr(),
                               err.data_ptr() if err is not None else None, _stream_ptr(stream))
    return logp


def gather_records(rec, group=None):
    """All-gather one rank's records [B, 4] into [P, B, 4] in rank order (the
    layout the merge calls read). torch.distributed provides the collective
    (NCCL between GPUs, gloo on CPU tensors)."""
    import torch
    import torch.distributed as dist
    P = dist.get_world_size(group)
    B = int(rec.shape[0])
    out = torch.empty((P * B,) + tuple(rec.shape[1:]), dtype=rec.dtype, device=rec.device)
    dist.all_gather_into_tensor(out, rec.contiguous(), group=group)
    return out.view((P, B) + tuple(rec.shape[1:]))


class VocabParallelHead:
    """The output head split by vocabulary over the ranks of a process group:
    rank r holds W rows detlm_shard_range(V, P, r). A call runs this rank's
    shard, all-gathers one 16-byte record per hidden row and merges them, so
    every rank returns the single-device head's outputs bit for bit."""

    def __init__(self, W_shard, V: int, group=None, dtype: str | None = None):
        import torch.distributed as dist
        self.group = group
        P, r = dist.get_world_size(group), dist.get_rank(group)
        self.shard = ShardHead(W_shard, V, P, r, dtype)

    def greedy(self, h, stream=None):
        rec, _ = self.shard.greedy_records(h, stream=stream)
        return merge_greedy(gather_records(rec, self.group), self.shard.dtype, stream=stream)

    def logprob(self, h, targets, stream=None):
        rec = self.shard.logprob_records(h, targets, stream=stream)
        return merge_logprob(gather_records(rec, self.group), self.shard.V_total, targets,
                             stream=stream)

    def close(self):
        self.shard.close()
