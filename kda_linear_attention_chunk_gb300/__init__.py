"""Python binding of libkda.so, the GB300 KDA chunked packed-varlen prefill.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI of include/kda.h.  PyTorch supplies device memory
and streams.  There is no fallback: if the library is not built, the entry
points raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkda.so")

KDA_OK, KDA_ERR_NULL, KDA_ERR_SHAPE, KDA_ERR_UNSUPPORTED = 0, 1, 2, 3
KDA_ERR_ALIGN, KDA_ERR_ALIAS, KDA_ERR_CUDA, KDA_ERR_DEVICE = 4, 5, 6, 7
KDA_ERR_NOALLOC_LIMIT = 8
KDA_NOALLOC_MAX_SEQS = 16384

EXPORTED = ("kda_chunk_prefill", "kda_chunk_prefill_f32", "kda_chunk_prefill_fullrange", "kda_status_string",
            "kda_device_error", "kda_chunk_prefill_noalloc", "kda_chunk_prefill_slots", "kda_chunk_prefill_conv",
            "kda_decode", "kda_fold_commit", "kda_short_conv", "kda_decode_conv", "kda_head_norm_rope",
            "kda_window_prefill", "kda_window_decode", "kda_slots_copy", "kda_slots_compact", "kda_paged_append",
            "kda_paged_attention", "kda_paged_attention_workspace", "kda_pages_copy", "kda_beam_select",
            "kda_beam_select_workspace")
# device error word bits (kda_device_error)
ERR_WAIT_TIMEOUT = 1    # a bounded wait ran out; the kernel wound down early
ERR_BAD_SEQLENS = 2     # a cu_seqlens entry broke its contract (clamped)
ERR_BAD_SLOT = 8        # a state slot id outside [-1, num_slots)
ERR_BAD_ACCEPTED = 16   # an accepted count outside [0, window]
ERR_DECAY_RANGE = 32    # the tensor-core prefill met a decay beyond its fp16 operand range
ERR_BAD_POSITION = 64   # a position or context length outside its range (clamped)
ERR_BAD_PAGE = 128      # a page id outside [0, num_pages) where a page was needed

KDA_BF16, KDA_F16, KDA_F32 = 0, 1, 2
KDA_ROPE_HALF, KDA_ROPE_INTERLEAVED = 0, 1
KDA_MAX_POOLS, KDA_MAX_POOL_SLOTS = 128, 524288

_lib = None
_torch_module = None


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}" if where else status_string(status))


def load(path: str = LIB_PATH):
    """Load libkda.so (built by __graft_entry__.build()); raises if missing."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libkda.so is not built ({path}); run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    P, I = ctypes.c_void_p, ctypes.c_int
    sig = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, P]
    for name in ("kda_chunk_prefill", "kda_chunk_prefill_f32", "kda_chunk_prefill_fullrange",
                 "kda_chunk_prefill_noalloc"):
        fn = getattr(lib, name)
        fn.argtypes = sig
        fn.restype = I
    lib.kda_chunk_prefill_slots.argtypes = [P, P, P, P, P, P, P, P, I, P, I, I, I, I, I, P]
    lib.kda_chunk_prefill_slots.restype = I
    lib.kda_chunk_prefill_conv.argtypes = [P, P, P, P, P, P, P, P, P, I, P, I, P, I, I, I, I, I, I,
                                           ctypes.c_float, P]
    lib.kda_chunk_prefill_conv.restype = I
    lib.kda_decode.argtypes = [P, P, P, P, P, P, P, I, P, I, I, I, I, P]
    lib.kda_decode.restype = I
    lib.kda_fold_commit.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P]
    lib.kda_fold_commit.restype = I
    lib.kda_short_conv.argtypes = [P, P, P, P, P, P, P, I, P, P, P, I, I, I, I, I, ctypes.c_float, P]
    lib.kda_short_conv.restype = I
    lib.kda_decode_conv.argtypes = [P, P, P, P, P, P, I, P, P, P, P, I, P, I, I, I, I, I, ctypes.c_float, P]
    lib.kda_decode_conv.restype = I
    L, F = ctypes.c_int64, ctypes.c_float
    lib.kda_head_norm_rope.argtypes = [P, L, P, L, P, P, P, I, P, P, P, I, I, I, I, I, I, I, F, I, P]
    lib.kda_window_prefill.argtypes = [P, L, P, L, P, L, P, P, P, P, I, I, P, I, I, I, I, I, I, I, F, I, P]
    lib.kda_window_decode.argtypes = [P, L, P, L, P, L, P, P, P, I, I, P, I, I, I, I, I, I, F, I, P]
    lib.kda_slots_copy.argtypes = [P, I, I, P, P, I, P]
    lib.kda_slots_compact.argtypes = [P, I, I, P, P, I, P]
    for name in ("kda_head_norm_rope", "kda_window_prefill", "kda_window_decode", "kda_slots_copy", "kda_slots_compact"):
        getattr(lib, name).restype = I
    lib.kda_paged_append.argtypes = [P, L, P, L, P, L, P, P, P, I, P, P, P, P, I, I, P, I, I, P, I, I, I, I, I, I, I, I, F,
                                     I, P]
    lib.kda_paged_attention.argtypes = [P, L, P, P, P, P, I, I, P, I, I, P, P, P, I, P, P, L, I, I, I, I, I, F, I, P]
    lib.kda_pages_copy.argtypes = [P, I, I, I, I, P, I, I, P, P, P, P, I, P]
    lib.kda_beam_select.argtypes = [P, L, I, P, P, I, P, P, P, P, P, P, P, P, P, L, I, I, I, P]
    for name in ("kda_paged_append", "kda_paged_attention", "kda_pages_copy", "kda_beam_select"):
        getattr(lib, name).restype = I
    lib.kda_paged_attention_workspace.argtypes = [I, I, I, I, I, I]
    lib.kda_beam_select_workspace.argtypes = [I, I, I]
    lib.kda_paged_attention_workspace.restype = lib.kda_beam_select_workspace.restype = L
    lib.kda_status_string.argtypes = [I]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_device_error.argtypes = [ctypes.POINTER(ctypes.c_int), I]
    lib.kda_device_error.restype = I
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().kda_status_string(int(status)).decode()
    except RuntimeError:
        return f"kda_status {status}"


def kda_chunk_prefill(q, k, v, g, beta, cu_seqlens, initial_state, out, final_state,
                      N: int, T: int, H: int, dk: int, dv: int, stream) -> int:
    """Raw C-ABI call: integer device pointers (0 = NULL) and sizes."""
    return load().kda_chunk_prefill(q, k, v, g, beta, cu_seqlens, initial_state, out, final_state,
                                    N, T, H, dk, dv, stream)


def kda_chunk_prefill_f32(q, k, v, g, beta, cu_seqlens, initial_state, out, final_state,
                          N: int, T: int, H: int, dk: int, dv: int, stream) -> int:
    """Raw C-ABI call for fp32 q/k/v/out."""
    return load().kda_chunk_prefill_f32(q, k, v, g, beta, cu_seqlens, initial_state, out,
                                        final_state, N, T, H, dk, dv, stream)


def kda_chunk_prefill_fullrange(q, k, v, g, beta, cu_seqlens, initial_state, out, final_state,
                                N: int, T: int, H: int, dk: int, dv: int, stream) -> int:
    """Raw C-ABI call of the bf16 prefill on the CUDA-core kernel, which takes
    any decay (no fp16 operand range)."""
    return load().kda_chunk_prefill_fullrange(q, k, v, g, beta, cu_seqlens, initial_state, out,
                                              final_state, N, T, H, dk, dv, stream)


def kda_chunk_prefill_noalloc(q, k, v, g, beta, cu_seqlens, initial_state, out, final_state,
                              N: int, T: int, H: int, dk: int, dv: int, stream) -> int:
    """Raw C-ABI call of the entry point that allocates nothing (up to
    KDA_NOALLOC_MAX_SEQS sequences; its scheduling table lives inside the
    library, for callers that cannot allocate device memory per call)."""
    return load().kda_chunk_prefill_noalloc(q, k, v, g, beta, cu_seqlens, initial_state, out,
                                            final_state, N, T, H, dk, dv, stream)


def kda_chunk_prefill_slots(q, k, v, g, beta, cu_seqlens, state_slots, state_pool, num_slots: int, out,
                            N: int, T: int, H: int, dk: int, dv: int, stream) -> int:
    """Raw C-ABI call with the states in a slot-addressed pool."""
    return load().kda_chunk_prefill_slots(q, k, v, g, beta, cu_seqlens, state_slots, state_pool,
                                          num_slots, out, N, T, H, dk, dv, stream)


def kda_chunk_prefill_conv(xq, xk, xv, conv_weight, g, beta, cu_seqlens, slots, conv_pool, conv_num_slots: int,
                           state_pool, num_slots: int, out, N: int, T: int, H: int, dk: int, dv: int,
                           activation: int, eps: float, stream) -> int:
    """Raw C-ABI call: the short-conv prologue fused into the prefill."""
    return load().kda_chunk_prefill_conv(xq, xk, xv, conv_weight, g, beta, cu_seqlens, slots, conv_pool,
                                         conv_num_slots, state_pool, num_slots, out, N, T, H, dk, dv, activation,
                                         eps, stream)


def kda_decode(q, k, v, g, beta, state_slots, state_pool, num_slots: int, out, N: int, H: int, dk: int, dv: int,
               stream) -> int:
    """Raw C-ABI call: one recurrence step per sequence on a slot-addressed pool."""
    return load().kda_decode(q, k, v, g, beta, state_slots, state_pool, num_slots, out, N, H, dk, dv, stream)


def kda_fold_commit(k, v, g, beta, accepted, state_slots, state_pool, num_slots: int, N: int, W: int, H: int,
                    dk: int, dv: int, stream) -> int:
    """Raw C-ABI call: fold the accepted tokens of each window into the pool."""
    return load().kda_fold_commit(k, v, g, beta, accepted, state_slots, state_pool, num_slots, N, W, H, dk, dv,
                                  stream)


def kda_short_conv(xq, xk, xv, conv_weight, cu_seqlens, conv_slots, conv_pool, num_slots: int, q_out, k_out,
                   v_out, N: int, T: int, H: int, d: int, activation: int, eps: float, stream) -> int:
    """Raw C-ABI call: short conv + L2 norm prologue, conv windows in a slot-addressed pool."""
    return load().kda_short_conv(xq, xk, xv, conv_weight, cu_seqlens, conv_slots, conv_pool, num_slots, q_out,
                                 k_out, v_out, N, T, H, d, activation, eps, stream)


def kda_decode_conv(xq, xk, xv, conv_weight, conv_slots, conv_pool, conv_num_slots: int, g, beta, state_slots,
                    state_pool, num_slots: int, out, N: int, H: int, dk: int, dv: int, activation: int, eps: float,
                    stream) -> int:
    """Raw C-ABI call: the decode step with the short conv fused in front of it."""
    return load().kda_decode_conv(xq, xk, xv, conv_weight, conv_slots, conv_pool, conv_num_slots, g, beta,
                                  state_slots, state_pool, num_slots, out, N, H, dk, dv, activation, eps, stream)


def kda_head_norm_rope(q, q_stride: int, k, k_stride: int, q_weight, k_weight, table, max_pos: int, positions, q_out,
                       k_out, T: int, Hq: int, Hk: int, d: int, rotary: int, layout: int, norm: int, eps: float,
                       dtype: int, stream) -> int:
    """Raw C-ABI call: per-head RMS norm and rotation of q and k."""
    return load().kda_head_norm_rope(q, q_stride, k, k_stride, q_weight, k_weight, table, max_pos, positions, q_out,
                                     k_out, T, Hq, Hk, d, rotary, layout, norm, eps, dtype, stream)


def kda_window_prefill(q, q_stride: int, k, k_stride: int, v, v_stride: int, cu_seqlens, starts, slots, kv_pool,
                       num_slots: int, pool_rows: int, out, N: int, T: int, Hq: int, Hk: int, d: int, window: int,
                       sinks: int, scale: float, dtype: int, stream) -> int:
    """Raw C-ABI call: window attention of packed new tokens over the ring cache and themselves."""
    return load().kda_window_prefill(q, q_stride, k, k_stride, v, v_stride, cu_seqlens, starts, slots, kv_pool,
                                     num_slots, pool_rows, out, N, T, Hq, Hk, d, window, sinks, scale, dtype, stream)


def kda_window_decode(q, q_stride: int, k, k_stride: int, v, v_stride: int, positions, slots, kv_pool,
                      num_slots: int, pool_rows: int, out, N: int, Hq: int, Hk: int, d: int, window: int, sinks: int,
                      scale: float, dtype: int, stream) -> int:
    """Raw C-ABI call: window attention of one new token per sequence over the ring cache."""
    return load().kda_window_decode(q, q_stride, k, k_stride, v, v_stride, positions, slots, kv_pool, num_slots,
                                    pool_rows, out, N, Hq, Hk, d, window, sinks, scale, dtype, stream)


def kda_slots_copy(pools, num_pools: int, num_slots: int, src, dst, M: int, stream) -> int:
    """Raw C-ABI call: copies (or clears) slot entries in every pool; pools is the address of a host array of
    (base, entry_bytes) pairs of 64-bit integers."""
    return load().kda_slots_copy(pools, num_pools, num_slots, src, dst, M, stream)


def kda_slots_compact(pools, num_pools: int, num_slots: int, slots, new_slots, N: int, stream) -> int:
    """Raw C-ABI call: moves the live slot entries to the front of every pool."""
    return load().kda_slots_compact(pools, num_pools, num_slots, slots, new_slots, N, stream)


def kda_paged_append(q, q_stride: int, k, k_stride: int, v, v_stride: int, q_weight, k_weight, table, max_pos: int,
                     cu_seqlens, starts, slots, kv_pages, num_pages: int, page: int, page_table, num_slots: int,
                     max_pages: int, q_out, N: int, T: int, Hq: int, Hk: int, d: int, rotary: int, layout: int, norm: int,
                     eps: float, dtype: int, stream) -> int:
    """Raw C-ABI call: norm and rotation of packed rows, k and v on their way into a paged cache."""
    return load().kda_paged_append(q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, table, max_pos, cu_seqlens,
                                   starts, slots, kv_pages, num_pages, page, page_table, num_slots, max_pages, q_out, N,
                                   T, Hq, Hk, d, rotary, layout, norm, eps, dtype, stream)


def kda_paged_attention(q, q_stride: int, cu_seqlens, starts, slots, kv_pages, num_pages: int, page: int, page_table,
                        num_slots: int, max_pages: int, groups, prefix_lens, prefix_slots, P: int, out, workspace,
                        workspace_bytes: int, N: int, T: int, Hq: int, Hk: int, d: int, scale: float, dtype: int,
                        stream) -> int:
    """Raw C-ABI call: causal attention of packed rows over a paged cache with shared prefixes."""
    return load().kda_paged_attention(q, q_stride, cu_seqlens, starts, slots, kv_pages, num_pages, page, page_table,
                                      num_slots, max_pages, groups, prefix_lens, prefix_slots, P, out, workspace,
                                      workspace_bytes, N, T, Hq, Hk, d, scale, dtype, stream)


def kda_paged_attention_workspace(N: int, T: int, P: int, Hq: int, Hk: int, d: int) -> int:
    """Raw C-ABI call: the workspace bytes of a kda_paged_attention call, -1 for sizes that none may have."""
    return load().kda_paged_attention_workspace(N, T, P, Hq, Hk, d)


def kda_pages_copy(caches, num_caches: int, num_pages: int, page: int, row_bytes: int, page_table, num_slots: int,
                   max_pages: int, src, dst, start, end, M: int, stream) -> int:
    """Raw C-ABI call: copies position ranges between slots in several paged caches; caches is the address of a host
    array of (base, bytes of a page) pairs of 64-bit integers."""
    return load().kda_pages_copy(caches, num_caches, num_pages, page, row_bytes, page_table, num_slots, max_pages, src,
                                 dst, start, end, M, stream)


def kda_beam_select(logits, row_stride: int, dtype: int, scores, ended, end_token: int, slots, scores_out, parents, tokens,
                    ended_out, new_slots, src, dst, workspace, workspace_bytes: int, G: int, B: int, V: int, stream) -> int:
    """Raw C-ABI call: one selection step of beam search."""
    return load().kda_beam_select(logits, row_stride, dtype, scores, ended, end_token, slots, scores_out, parents, tokens,
                                  ended_out, new_slots, src, dst, workspace, workspace_bytes, G, B, V, stream)


def kda_beam_select_workspace(G: int, B: int, V: int) -> int:
    """Raw C-ABI call: the workspace bytes of a kda_beam_select call, -1 for sizes that none may have."""
    return load().kda_beam_select_workspace(G, B, V)


def device_error(reset: bool = False) -> int:
    word = ctypes.c_int(0)
    st = load().kda_device_error(ctypes.byref(word), int(reset))
    if st != KDA_OK:
        raise KdaError(st, "kda_device_error")
    return word.value


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def chunk_prefill(q, k, v, g, beta, cu_seqlens, initial_state=None, out=None, final_state=None,
                  output_final_state: bool = True, stream=None,
                  full_range: bool = False) -> Tuple[object, Optional[object]]:
    """KDA chunked packed-varlen prefill on torch CUDA tensors.

    q, k: [T][H][dk], v: [T][H][dv] (bfloat16 or float32; dk, dv in {64, 128});
    g: [T][H][dk] float32; beta: [T][H] float32; cu_seqlens: [N+1] int32 on
    the device; initial_state: [N][H][dv][dk] float32 or None.  Returns
    (out [T][H][dv] in q's dtype, final_state [N][H][dv][dk] float32 or None).
    Runs asynchronously on ``stream`` (default: torch's current stream).
    ``full_range`` (bfloat16 only) selects kda_chunk_prefill_fullrange, for
    decays beyond the tensor-core kernel's range (ERR_DECAY_RANGE).
    """
    import torch

    T, H, dk = q.shape
    dv = v.shape[2]
    N = cu_seqlens.shape[0] - 1
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("cu_seqlens", cu_seqlens)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if out is None:
        out = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    s = stream if stream is not None else torch.cuda.current_stream(q.device)
    handle = int(s.cuda_stream) if hasattr(s, "cuda_stream") else int(s)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(initial_state),
            _ptr(out), _ptr(final_state), N, T, H, dk, dv, handle)
    if q.dtype == torch.bfloat16:
        st = kda_chunk_prefill_fullrange(*args) if full_range else kda_chunk_prefill(*args)
    elif q.dtype == torch.float32:
        st = kda_chunk_prefill_f32(*args)
    else:
        raise ValueError(f"unsupported q dtype {q.dtype}")
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_prefill")
    return out, final_state


def chunk_prefill_slots(q, k, v, g, beta, cu_seqlens, state_slots, state_pool, out=None, stream=None):
    """KDA prefill with slot-addressed states, on torch CUDA tensors.

    q, k, v: [T][H][128] bfloat16; g: [T][H][128] float32; beta: [T][H]
    float32; cu_seqlens: [N+1] int32 and state_slots: [N] int32 on the device
    (-1 = padded sequence, skipped); state_pool: [num_slots][H][128][128]
    float32, read and updated in place.  Returns out [T][H][128] bfloat16
    (rows of padded sequences keep what ``out`` held; a fresh ``out`` is
    uninitialised there).  Runs asynchronously on ``stream``.
    """
    import torch

    T, H, dk = q.shape
    dv = v.shape[2]
    N = cu_seqlens.shape[0] - 1
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("cu_seqlens", cu_seqlens),
                    ("state_slots", state_slots), ("state_pool", state_pool)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if q.dtype != torch.bfloat16:
        raise ValueError("chunk_prefill_slots takes bfloat16 q/k/v")
    if state_slots.dtype != torch.int32 or tuple(state_slots.shape) != (N,):
        raise ValueError("state_slots must be int32 [N]")
    if state_pool.dtype != torch.float32 or tuple(state_pool.shape[1:]) != (H, dv, dk):
        raise ValueError("state_pool must be float32 [num_slots][H][dv][dk]")
    if out is None:
        out = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    s = stream if stream is not None else torch.cuda.current_stream(q.device)
    handle = int(s.cuda_stream) if hasattr(s, "cuda_stream") else int(s)
    st = kda_chunk_prefill_slots(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                 _ptr(state_slots), _ptr(state_pool), int(state_pool.shape[0]), _ptr(out),
                                 N, T, H, dk, dv, handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_prefill_slots")
    return out


def decode(q, k, v, g, beta, state_pool, state_slots=None, out=None, stream=None):
    """One KDA recurrence step per sequence (decode) on torch CUDA tensors.

    q, k, v: [N][H][128] bfloat16 (row n = sequence n's new token); g:
    [N][H][128] float32; beta: [N][H] float32; state_pool:
    [num_slots][H][128][128] float32, updated in place; state_slots: [N] int32
    on the device (-1 = padded row, skipped) or None for entry n.  Returns out
    [N][H][128] bfloat16 (rows of padded sequences keep what ``out`` held).
    """
    import torch

    N, H, dk = q.shape
    dv = v.shape[2]
    tensors = [("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("state_pool", state_pool)]
    if state_slots is not None:
        tensors.append(("state_slots", state_slots))
    for name, t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if q.dtype != torch.bfloat16:
        raise ValueError("decode takes bfloat16 q/k/v")
    if state_slots is not None and (state_slots.dtype != torch.int32 or tuple(state_slots.shape) != (N,)):
        raise ValueError("state_slots must be int32 [N]")
    if state_pool.dtype != torch.float32 or tuple(state_pool.shape[1:]) != (H, dv, dk):
        raise ValueError("state_pool must be float32 [num_slots][H][dv][dk]")
    if out is None:
        out = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    s = stream if stream is not None else torch.cuda.current_stream(q.device)
    handle = int(s.cuda_stream) if hasattr(s, "cuda_stream") else int(s)
    st = kda_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_slots), _ptr(state_pool),
                    int(state_pool.shape[0]), _ptr(out), N, H, dk, dv, handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_decode")
    return out


def fold_commit(k, v, g, beta, accepted, state_pool, state_slots=None, stream=None):
    """Commit of a speculative round on torch CUDA tensors: the first accepted[n]
    tokens of sequence n's window are folded into its state.

    k, v: [N][W][H][128] bfloat16; g: [N][W][H][128] float32; beta: [N][W][H]
    float32; accepted: [N] int32 on the device; state_pool:
    [num_slots][H][128][128] float32, updated in place; state_slots: [N] int32
    (-1 = skip) or None for entry n.
    """
    import torch

    N, W, H, dk = k.shape
    dv = v.shape[3]
    tensors = [("k", k), ("v", v), ("g", g), ("beta", beta), ("accepted", accepted), ("state_pool", state_pool)]
    if state_slots is not None:
        tensors.append(("state_slots", state_slots))
    for name, t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if k.dtype != torch.bfloat16:
        raise ValueError("fold_commit takes bfloat16 k/v")
    if accepted.dtype != torch.int32 or tuple(accepted.shape) != (N,):
        raise ValueError("accepted must be int32 [N]")
    if state_pool.dtype != torch.float32 or tuple(state_pool.shape[1:]) != (H, dv, dk):
        raise ValueError("state_pool must be float32 [num_slots][H][dv][dk]")
    s = stream if stream is not None else torch.cuda.current_stream(k.device)
    handle = int(s.cuda_stream) if hasattr(s, "cuda_stream") else int(s)
    st = kda_fold_commit(_ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(accepted), _ptr(state_slots),
                         _ptr(state_pool), int(state_pool.shape[0]), N, W, H, dk, dv, handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_fold_commit")


ACTIVATIONS = {"none": 0, "silu": 1}


def short_conv(xq, xk, xv, conv_weight, cu_seqlens, conv_pool, conv_slots=None, activation: str = "silu",
               eps: float = 1e-6, out=None, stream=None):
    """Short conv + L2 norm prologue on torch CUDA tensors.

    xq, xk, xv: [T][H][128] bfloat16; conv_weight: [3][H*128][4] float32 (tap
    3 weighs the row itself); cu_seqlens: [N+1] int32; conv_pool:
    [num_slots][3][3][H*128] bfloat16, updated in place; conv_slots: [N] int32
    (-1 = padded, skipped) or None for entry n.  activation "none" or "silu".
    Returns (q, k, v), each [T][H][128] bfloat16 (q and k with unit L2 norm
    per head).
    """
    import torch

    T, H, d = xq.shape
    N = int(cu_seqlens.shape[0]) - 1
    tensors = [("xq", xq), ("xk", xk), ("xv", xv), ("conv_weight", conv_weight), ("cu_seqlens", cu_seqlens),
               ("conv_pool", conv_pool)]
    if conv_slots is not None:
        tensors.append(("conv_slots", conv_slots))
    for name, t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if xq.dtype != torch.bfloat16 or xk.dtype != torch.bfloat16 or xv.dtype != torch.bfloat16:
        raise ValueError("short_conv takes bfloat16 projections")
    if conv_weight.dtype != torch.float32 or tuple(conv_weight.shape) != (3, H * d, 4):
        raise ValueError("conv_weight must be float32 [3][H*d][4]")
    if conv_pool.dtype != torch.bfloat16 or tuple(conv_pool.shape[1:]) != (3, 3, H * d):
        raise ValueError("conv_pool must be bfloat16 [num_slots][3][3][H*d]")
    if conv_slots is not None and (conv_slots.dtype != torch.int32 or tuple(conv_slots.shape) != (N,)):
        raise ValueError("conv_slots must be int32 [N]")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    if out is None:
        out = tuple(torch.empty_like(xq) for _ in range(3))
    q, k, v = out
    s = stream if stream is not None else torch.cuda.current_stream(xq.device)
    handle = int(s.cuda_stream) if hasattr(s, "cuda_stream") else int(s)
    st = kda_short_conv(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(conv_weight), _ptr(cu_seqlens), _ptr(conv_slots),
                        _ptr(conv_pool), int(conv_pool.shape[0]), _ptr(q), _ptr(k), _ptr(v), N, T, H, d,
                        ACTIVATIONS[activation], float(eps), handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_short_conv")
    return q, k, v


def chunk_prefill_conv(xq, xk, xv, conv_weight, g, beta, cu_seqlens, conv_pool, state_pool, slots=None,
                       activation: str = "silu", eps: float = 1e-6, out=None, stream=None):
    """A KDA layer's prefill with the short-conv + L2-norm prologue fused in,
    on torch CUDA tensors.

    xq, xk, xv: [T][H][128] bfloat16 projections; conv_weight: [3][H*128][4]
    float32; g: [T][H][128] float32; beta: [T][H] float32; cu_seqlens: [N+1]
    int32; conv_pool: [conv_num_slots][3][3][H*128] bfloat16 and state_pool:
    [num_slots][H][128][128] float32, both updated in place; slots: [N] int32
    (-1 = padded, skipped) or None for entry n of both pools.  Returns out
    [T][H][128] bfloat16 (rows of padded sequences keep what ``out`` held).
    """
    import torch

    T, H, d = xq.shape
    N = int(cu_seqlens.shape[0]) - 1
    tensors = [("xq", xq), ("xk", xk), ("xv", xv), ("conv_weight", conv_weight), ("g", g), ("beta", beta),
               ("cu_seqlens", cu_seqlens), ("conv_pool", conv_pool), ("state_pool", state_pool)]
    if slots is not None:
        tensors.append(("slots", slots))
        if slots.dtype != torch.int32 or tuple(slots.shape) != (N,):
            raise ValueError("slots must be int32 [N]")
    for name, t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if xq.dtype != torch.bfloat16 or xk.dtype != torch.bfloat16 or xv.dtype != torch.bfloat16:
        raise ValueError("chunk_prefill_conv takes bfloat16 projections")
    if conv_weight.dtype != torch.float32 or tuple(conv_weight.shape) != (3, H * d, 4):
        raise ValueError("conv_weight must be float32 [3][H*d][4]")
    if conv_pool.dtype != torch.bfloat16 or tuple(conv_pool.shape[1:]) != (3, 3, H * d):
        raise ValueError("conv_pool must be bfloat16 [num_slots][3][3][H*d]")
    if state_pool.dtype != torch.float32 or tuple(state_pool.shape[1:]) != (H, d, d):
        raise ValueError("state_pool must be float32 [num_slots][H][d][d]")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    if out is None:
        out = torch.empty((T, H, d), dtype=xq.dtype, device=xq.device)
    s = stream if stream is not None else torch.cuda.current_stream(xq.device)
    handle = int(s.cuda_stream) if hasattr(s, "cuda_stream") else int(s)
    st = kda_chunk_prefill_conv(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(conv_weight), _ptr(g), _ptr(beta),
                                _ptr(cu_seqlens), _ptr(slots), _ptr(conv_pool), int(conv_pool.shape[0]),
                                _ptr(state_pool), int(state_pool.shape[0]), _ptr(out), N, T, H, d, d,
                                ACTIVATIONS[activation], float(eps), handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_prefill_conv")
    return out


def decode_conv(xq, xk, xv, conv_weight, conv_pool, g, beta, state_pool, conv_slots=None, state_slots=None,
                activation: str = "silu", eps: float = 1e-6, out=None, stream=None):
    """The decode step with the short conv + L2 norm prologue fused in front of
    it, on torch CUDA tensors.

    xq, xk, xv: [N][H][128] bfloat16 (row n = sequence n's new token, before
    the conv); conv_weight: [3][H*128][4] float32; conv_pool:
    [conv_num_slots][3][3][H*128] bfloat16 and state_pool:
    [num_slots][H][128][128] float32, both updated in place; conv_slots,
    state_slots: [N] int32 (-1 = padded row, skipped) or None for entry n;
    g: [N][H][128] float32; beta: [N][H] float32.  Returns out [N][H][128]
    bfloat16 (rows of padded sequences keep what ``out`` held).
    """
    import torch

    N, H, d = xq.shape
    tensors = [("xq", xq), ("xk", xk), ("xv", xv), ("conv_weight", conv_weight), ("conv_pool", conv_pool),
               ("g", g), ("beta", beta), ("state_pool", state_pool)]
    for name, t in (("conv_slots", conv_slots), ("state_slots", state_slots)):
        if t is not None:
            tensors.append((name, t))
            if t.dtype != torch.int32 or tuple(t.shape) != (N,):
                raise ValueError(f"{name} must be int32 [N]")
    for name, t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if xq.dtype != torch.bfloat16 or xk.dtype != torch.bfloat16 or xv.dtype != torch.bfloat16:
        raise ValueError("decode_conv takes bfloat16 projections")
    if conv_weight.dtype != torch.float32 or tuple(conv_weight.shape) != (3, H * d, 4):
        raise ValueError("conv_weight must be float32 [3][H*d][4]")
    if conv_pool.dtype != torch.bfloat16 or tuple(conv_pool.shape[1:]) != (3, 3, H * d):
        raise ValueError("conv_pool must be bfloat16 [num_slots][3][3][H*d]")
    if state_pool.dtype != torch.float32 or tuple(state_pool.shape[1:]) != (H, d, d):
        raise ValueError("state_pool must be float32 [num_slots][H][dv][dk]")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    if out is None:
        out = torch.empty((N, H, d), dtype=xq.dtype, device=xq.device)
    s = stream if stream is not None else torch.cuda.current_stream(xq.device)
    handle = int(s.cuda_stream) if hasattr(s, "cuda_stream") else int(s)
    st = kda_decode_conv(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(conv_weight), _ptr(conv_slots), _ptr(conv_pool),
                         int(conv_pool.shape[0]), _ptr(g), _ptr(beta), _ptr(state_slots), _ptr(state_pool),
                         int(state_pool.shape[0]), _ptr(out), N, H, d, d, ACTIVATIONS[activation], float(eps),
                         handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_conv")
    return out


ROPE_LAYOUTS = {"half": KDA_ROPE_HALF, "interleaved": KDA_ROPE_INTERLEAVED}


def _torch():
    """The torch module, imported by the first call that needs it (a later import statement looks it up anew, and a call
    on small tensors is all host time)."""
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _current_device() -> int:
    return _torch()._C._cuda_getDevice()


def _device_of(name: str, t) -> int:
    """The index of the device of a call's first tensor.  The library launches on the current device with the addresses
    that it gets, so it has to be that one, and the other tensors and the stream have to be the device's too."""
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if at != _current_device():
        raise ValueError(f"{name} lies on cuda:{at}, which is not the current device")
    return at


def _handle(stream, device) -> int:
    """The stream's handle; without one, torch's current stream of the device (its raw handle: building a Stream object
    for it would cost as much as the rest of a call)."""
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(device.index)
    if getattr(stream, "device_index", device.index) != device.index:
        raise ValueError(f"the stream is not one of {device}")
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _new(shape, dtype, device, stream):
    """An output of a call on ``stream``.  Its memory has to be free on that stream, whatever torch's current stream still
    does with blocks it has given back; and it is not given back before the current stream, where it will be used, is
    done with it."""
    torch = _torch()
    if stream is None or _handle(stream, device) == _handle(None, device):
        return torch.empty(shape, dtype=dtype, device=device)
    current, handle = torch.cuda.current_stream(device), _handle(stream, device)
    # the default stream's handles (0, and 1 by name) are none that ExternalStream takes
    given = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    with torch.cuda.stream(given):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(current)
    return out


def _scratch(size: int, device, stream):
    """A workspace of a call on ``stream``: its memory belongs to that stream, so a later call on the stream may get it
    again, and none on another."""
    torch = _torch()
    if stream is None or _handle(stream, device) == _handle(None, device):
        return torch.empty(size, dtype=torch.uint8, device=device)
    handle = _handle(stream, device)
    given = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    with torch.cuda.stream(given):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _dtype16(t, name: str) -> int:
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return KDA_BF16
    if t.dtype is torch.float16:
        return KDA_F16
    raise ValueError(f"{name} must be bfloat16 or float16")


def _rows_of_heads(name: str, t, dtype, at: int):
    """Checks rows of [heads][d] dense elements on device ``at``; returns the shape and the rows' distance in elements."""
    if t.get_device() != at or t.dim() != 3 or t.dtype != dtype:
        raise ValueError(f"{name} must be a tensor [rows][heads][d] of q's dtype and device")
    n, h, d = shape = t.shape
    row, head, one = t.stride()
    if one != 1 or (h > 1 and head != d):
        raise ValueError(f"{name} must be dense within each row")
    return shape, row if n > 1 else h * d


def _table32(name: str, t, n: int, at: int) -> int:
    """Checks an int32 [n] table on device ``at``; returns its address."""
    if t.dtype is not _torch().int32 or t.get_device() != at or not t.is_contiguous() or t.shape != (n,):
        raise ValueError(f"{name} must be int32 [{n}] on the device")
    return t.data_ptr()


def _dense(name: str, t, shape, dtype, at: int) -> int:
    """Checks a contiguous tensor on device ``at``; returns its address."""
    if t.dtype != dtype or t.get_device() != at or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name} must be a contiguous tensor {list(shape)} of {dtype} on the device")
    return t.data_ptr()


def rope_table(max_pos: int, rotary: int, base: float = 10000.0, stretch: float = 1.0, trained: int = 0,
               fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Cosines and sines of the positions 0 .. max_pos-1 for head_norm_rope: float32 [max_pos][rotary], computed in
    float64.  Pair i of a head turns by base^(-2i/rotary) per position.

    A context ``stretch`` times the trained one: with ``trained`` 0 every frequency is divided by ``stretch``
    (positions are interpolated).  With ``trained`` the trained context's length, frequencies are interpolated by
    parts (the YaRN method): a pair that turns at least ``fast`` times within the trained context keeps its
    frequency, one that turns at most ``slow`` times has it divided, those between are blended linearly in the pair's
    index, and the table is scaled by 1 + 0.1 ln(stretch), so that logits grow with its square.
    """
    import math

    import torch

    if max_pos < 1 or rotary < 2 or rotary % 2 or not base > 1.0 or not stretch >= 1.0 or trained < 0:
        raise ValueError("rope_table needs max_pos >= 1, an even rotary >= 2, base > 1, stretch >= 1, trained >= 0")
    i = torch.arange(rotary // 2, dtype=torch.float64, device=device)
    f = base ** (-2.0 * i / rotary)
    size = 1.0
    if trained and stretch > 1.0:
        def pair_of(turns):   # the (real-valued) pair that turns so often within the trained context
            return rotary * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        lo, hi = max(0.0, math.floor(pair_of(fast))), min(rotary - 1.0, math.ceil(pair_of(slow)))
        part = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        f = f * (1.0 - part) + f / stretch * part
        size = 1.0 + 0.1 * math.log(stretch)
    else:
        f = f / stretch
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).mul_(size).float()


def head_norm_rope(q, k, q_weight=None, k_weight=None, positions=None, table=None, layout: str = "half",
                   eps: float = 1e-6, norm: bool = True, out=None, stream=None):
    """Per-head RMS norm and rotation of q and k in one pass, on torch CUDA tensors.

    q: [T][Hq][d], k: [T][Hk][d], bfloat16 or float16, d 64 or 128, dense within a row (rows may be slices of a fused
    projection); q_weight, k_weight: [d] float32 or None; table: [max_pos][rotary] float32 (rope_table) with positions: [T]
    int32, or None (no rotation); layout "half" or "interleaved".  ``norm`` False rotates only.  Returns
    (q, k), dense; ``out`` may name them (in place where the inputs are dense).
    """
    torch = _torch()
    dtype = q.dtype
    dt, at = _dtype16(q, "q"), _device_of("q", q)
    (T, Hq, d), sq = _rows_of_heads("q", q, dtype, at)
    k_shape, sk = _rows_of_heads("k", k, dtype, at)
    Hk = k_shape[1]
    if k_shape != (T, Hk, d):
        raise ValueError("k must have q's rows and head size")
    qw = kw = tab = pos = rotary = max_pos = 0
    if q_weight is not None:
        qw = _dense("q_weight", q_weight, (d,), torch.float32, at)
    if k_weight is not None:
        kw = _dense("k_weight", k_weight, (d,), torch.float32, at)
    if table is not None:
        if positions is None:
            raise ValueError("a table needs positions")
        if table.dim() != 2:
            raise ValueError("table must be [max_pos][rotary]")
        max_pos, rotary = shape = table.shape
        tab = _dense("table", table, shape, torch.float32, at)
        pos = _table32("positions", positions, T, at)
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    if out is None:
        q_out = _new((T, Hq, d), dtype, q.device, stream)
        k_out = _new(k_shape, dtype, q.device, stream)
    else:
        q_out, k_out = out
        _dense("out[0]", q_out, (T, Hq, d), dtype, at)
        _dense("out[1]", k_out, k_shape, dtype, at)
    st = load().kda_head_norm_rope(q.data_ptr(), sq, k.data_ptr(), sk, qw, kw, tab, max_pos, pos, q_out.data_ptr(),
                                   k_out.data_ptr(), T, Hq, Hk, d, rotary, ROPE_LAYOUTS[layout], 1 if norm else 0, eps,
                                   dt, _handle(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_head_norm_rope")
    return q_out, k_out


def _window_args(q, k, v, kv_pool, slots, N, out, window, sinks, stream):
    """The checks that the two window-attention calls share; returns what both pass on."""
    if not 0 < window <= 0x7fffffff or not 0 <= sinks <= 0x7fffffff:
        raise ValueError("window and sinks must be 32-bit numbers, window >= 1, sinks >= 0")
    dtype = q.dtype
    dt, at = _dtype16(q, "q"), _device_of("q", q)
    (T, Hq, d), sq = _rows_of_heads("q", q, dtype, at)
    k_shape, sk = _rows_of_heads("k", k, dtype, at)
    v_shape, sv = _rows_of_heads("v", v, dtype, at)
    Hk = k_shape[1]
    if k_shape != (T, Hk, d) or v_shape != k_shape:
        raise ValueError("k and v must have q's rows and head size, and the same heads")
    num_slots = rows = pool = 0
    if kv_pool is not None:
        if kv_pool.dim() != 5:
            raise ValueError("kv_pool must be [num_slots][2][Hk][rows][d]")
        num_slots, _, _, rows, _ = kv_pool.shape
        if not num_slots or not rows:            # its null address would stand for no cache
            raise ValueError("kv_pool has no entry")
        pool = _dense("kv_pool", kv_pool, (num_slots, 2, Hk, rows, d), dtype, at)
    ids = 0 if slots is None else _table32("slots", slots, N, at)
    if out is None:
        out = _new((T, Hq, d), dtype, q.device, stream)
    else:
        _dense("out", out, (T, Hq, d), dtype, at)
    return dt, at, (q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv), ids, (pool, num_slots, rows), out, T, Hq, Hk, d


def window_prefill(q, k, v, cu_seqlens, window: int, sinks: int = 0, kv_pool=None, slots=None, starts=None,
                   scale: Optional[float] = None, out=None, stream=None):
    """Attention of packed new tokens over a sliding window and the first ``sinks`` positions, on torch CUDA tensors.

    q: [T][Hq][d], k, v: [T][Hk][d], bfloat16 or float16, d 64 or 128, dense within a row; cu_seqlens: [N+1] int32 on
    the device; kv_pool: [num_slots][2][Hk][rows][d], the ring caches (rows >= sinks + window), read and updated in
    place, or None (nothing cached); slots: [N] int32 (-1 = padded sequence, skipped) or None for entry n; starts: [N]
    int32, the tokens of each sequence already cached, or None for 0; scale: d^-0.5 by default.  Returns out
    [T][Hq][d] (rows of padded sequences keep what ``out`` held).
    """
    N = int(cu_seqlens.shape[0]) - 1
    dt, at, qkv, ids, pool, out, T, Hq, Hk, d = _window_args(q, k, v, kv_pool, slots, N, out, window, sinks, stream)
    cu = _table32("cu_seqlens", cu_seqlens, N + 1, at)
    st = load().kda_window_prefill(*qkv, cu, 0 if starts is None else _table32("starts", starts, N, at), ids, *pool,
                                   out.data_ptr(), N, T, Hq, Hk, d, window, sinks, d ** -0.5 if scale is None else scale,
                                   dt, _handle(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_window_prefill")
    return out


def window_decode(q, k, v, positions, kv_pool, window: int, sinks: int = 0, slots=None,
                  scale: Optional[float] = None, out=None, stream=None):
    """window_prefill for one new token per sequence, on torch CUDA tensors: row n of q [N][Hq][d], k and v
    [N][Hk][d] is at position positions[n] ([N] int32 on the device, the tokens cached before it); k and v enter
    kv_pool in place.  Returns out [N][Hq][d] (rows of padded sequences, slot -1, keep what ``out`` held).
    """
    N = q.shape[0]
    dt, at, qkv, ids, pool, out, _, Hq, Hk, d = _window_args(q, k, v, kv_pool, slots, N, out, window, sinks, stream)
    st = load().kda_window_decode(*qkv, _table32("positions", positions, N, at), ids, *pool, out.data_ptr(), N, Hq, Hk, d,
                                  window, sinks, d ** -0.5 if scale is None else scale, dt, _handle(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_window_decode")
    return out


def _pools(pools):
    """A host array of (base, entry_bytes) pairs, the number of slots and the device of a list of pool tensors."""
    if not pools:
        raise ValueError("at least one pool is needed")
    at = _device_of("pools[0]", pools[0])
    n = pools[0].shape[0] if pools[0].dim() else 0
    flat = []
    for p in pools:
        if p.get_device() != at or not p.is_contiguous() or p.dim() < 2 or p.shape[0] != n or not p.numel():
            raise ValueError("every pool must be a contiguous tensor [num_slots][...] of the same num_slots and device")
        flat += (p.data_ptr(), p.numel() // n * p.element_size())   # (the stride of an axis of one may be anything)
    return (ctypes.c_int64 * len(flat))(*flat), n, pools[0].device


def slots_copy(pools, src, dst, stream=None) -> None:
    """Copies slot entries in every pool of a list at once, on torch CUDA tensors: entry dst[i] becomes entry src[i],
    or zeros where src[i] is -1; dst[i] = -1 skips a row.  pools: contiguous [num_slots][...] tensors; src, dst: [M]
    int32 on the device (targets distinct and no other row's source).  Without rows nothing is done.
    """
    array, n, device = _pools(pools)
    at = device.index
    M = int(src.shape[0])
    ids = _table32("src", src, M, at), _table32("dst", dst, M, at)
    if not M:
        return
    st = load().kda_slots_copy(ctypes.addressof(array), len(pools), n, *ids, M, _handle(stream, device))
    if st != KDA_OK:
        raise KdaError(st, "kda_slots_copy")


def slots_compact(pools, slots, new_slots=None, stream=None):
    """Moves the live entries (slots[i] >= 0, each once) to the front of every pool of a list, on torch CUDA tensors:
    with m live entries, ids from m on take the free ids below m, both in ascending order.  slots: [N] int32 on the
    device.  Returns new_slots [N] int32, where each went (-1 stays).
    """
    array, n, device = _pools(pools)
    at = device.index
    N = int(slots.shape[0])
    _table32("slots", slots, N, at)
    if new_slots is None:
        new_slots = _new((N,), _torch().int32, device, stream)
    else:
        _table32("new_slots", new_slots, N, at)
    if not N:
        return new_slots
    st = load().kda_slots_compact(ctypes.addressof(array), len(array) // 2, n, _ptr(slots), _ptr(new_slots), N,
                                  _handle(stream, device))
    if st != KDA_OK:
        raise KdaError(st, "kda_slots_compact")
    return new_slots


def _paged(kv_pages, page_table, dtype, Hk, d, at: int):
    """Checks a paged cache and its page table; returns what the calls pass on of them."""
    if kv_pages.dim() != 5 or not kv_pages.numel():
        raise ValueError("kv_pages must be [num_pages][2][Hk][page][d]")
    num_pages, _, heads, page, _ = kv_pages.shape
    if page_table.dim() != 2 or not page_table.numel():
        raise ValueError("page_table must be [num_slots][max_pages]")
    pages = _dense("kv_pages", kv_pages, (num_pages, 2, heads if Hk is None else Hk, page, d), dtype, at)
    num_slots, max_pages = shape = page_table.shape
    return pages, num_pages, page, _dense("page_table", page_table, shape, _torch().int32, at), num_slots, max_pages


def _packed(cu_seqlens, starts, slots, T: int, at: int):
    """Checks the tables of packed rows (or, without cu_seqlens, of a row each); returns N and their addresses."""
    N = T if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    return (N, 0 if cu_seqlens is None else _table32("cu_seqlens", cu_seqlens, N + 1, at),
            0 if starts is None else _table32("starts", starts, N, at),
            0 if slots is None else _table32("slots", slots, N, at))


def paged_append(q, k, v, kv_pages, page_table, starts=None, cu_seqlens=None, slots=None, q_weight=None, k_weight=None,
                 table=None, layout: str = "half", eps: float = 1e-6, norm: bool = True, out=None, stream=None):
    """head_norm_rope of new rows with k and v on their way into a paged cache, on torch CUDA tensors.

    q: [T][Hq][d], k, v: [T][Hk][d], bfloat16 or float16, d 64 or 128, dense within a row; kv_pages:
    [num_pages][2][Hk][page][d], updated in place, with page_table: [num_slots][max_pages] int32 (position p of a slot is
    row p % page of page page_table[slot][p // page]); starts: [N] int32, the position of each sequence's first row, or
    None (0); cu_seqlens: [N+1] int32, or None (a row for each sequence); slots: [N] int32 (-1 = padded sequence, skipped)
    or None for table row n; q_weight, k_weight, table (rope_table), layout, eps, norm as for head_norm_rope, the
    positions being the cache's.  Returns q, dense (rows of padded sequences keep what ``out`` held; ``out`` may be a
    dense q).
    """
    torch = _torch()
    dtype = q.dtype
    dt, at = _dtype16(q, "q"), _device_of("q", q)
    (T, Hq, d), sq = _rows_of_heads("q", q, dtype, at)
    k_shape, sk = _rows_of_heads("k", k, dtype, at)
    v_shape, sv = _rows_of_heads("v", v, dtype, at)
    Hk = k_shape[1]
    if k_shape != (T, Hk, d) or v_shape != k_shape:
        raise ValueError("k and v must have q's rows and head size, and the same heads")
    cache = _paged(kv_pages, page_table, dtype, Hk, d, at)
    N, cu, first, ids = _packed(cu_seqlens, starts, slots, T, at)
    qw = kw = tab = rotary = max_pos = 0
    if q_weight is not None:
        qw = _dense("q_weight", q_weight, (d,), torch.float32, at)
    if k_weight is not None:
        kw = _dense("k_weight", k_weight, (d,), torch.float32, at)
    if table is not None:
        if table.dim() != 2:
            raise ValueError("table must be [max_pos][rotary]")
        max_pos, rotary = shape = table.shape
        tab = _dense("table", table, shape, torch.float32, at)
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    if out is None:
        out = _new((T, Hq, d), dtype, q.device, stream)
    else:
        _dense("out", out, (T, Hq, d), dtype, at)
    if not T:
        return out
    st = load().kda_paged_append(q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, qw, kw, tab, max_pos, cu, first, ids,
                                 *cache, out.data_ptr(), N, T, Hq, Hk, d, rotary, ROPE_LAYOUTS[layout], 1 if norm else 0,
                                 eps, dt, _handle(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_paged_append")
    return out


def paged_attention(q, kv_pages, page_table, starts=None, cu_seqlens=None, slots=None, prefixes=None,
                    scale: Optional[float] = None, out=None, stream=None):
    """Causal attention of new rows over a paged cache that holds their keys and values already (paged_append), on torch
    CUDA tensors.

    q: [T][Hq][d], bfloat16 or float16, d 64 or 128, dense within a row; kv_pages, page_table, starts, cu_seqlens and
    slots as for paged_append; scale: d^-0.5 by default.  ``prefixes`` (groups [P+1], lengths [P], slots [P], int32 on the
    device): the sequences groups[g] .. groups[g+1]-1 share their first lengths[g] positions, which are kept (and read)
    once, in the pages of slots[g] (-1: no prefix); their own pages hold the positions from there on.  Returns out
    [T][Hq][d] (rows of padded sequences keep what ``out`` held).
    """
    dtype = q.dtype
    dt, at = _dtype16(q, "q"), _device_of("q", q)
    (T, Hq, d), sq = _rows_of_heads("q", q, dtype, at)
    cache = _paged(kv_pages, page_table, dtype, None, d, at)
    Hk = kv_pages.shape[2]
    N, cu, first, ids = _packed(cu_seqlens, starts, slots, T, at)
    P = groups = lens = kept = 0
    if prefixes is not None:
        P = int(prefixes[1].shape[0])
        groups = _table32("prefixes[0]", prefixes[0], P + 1, at)
        lens, kept = _table32("prefixes[1]", prefixes[1], P, at), _table32("prefixes[2]", prefixes[2], P, at)
        if not P:
            groups = lens = kept = 0
    if out is None:
        out = _new((T, Hq, d), dtype, q.device, stream)
    else:
        _dense("out", out, (T, Hq, d), dtype, at)
    if not T:
        return out
    lib = load()
    size = lib.kda_paged_attention_workspace(N, T, P, Hq, Hk, d)
    work = _scratch(size, q.device, stream) if size > 0 else None
    st = lib.kda_paged_attention(q.data_ptr(), sq, cu, first, ids, *cache, groups, lens, kept, P, out.data_ptr(),
                                 0 if work is None else work.data_ptr(), size, N, T, Hq, Hk, d,
                                 d ** -0.5 if scale is None else scale, dt, _handle(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_paged_attention")
    return out


def pages_copy(caches, page_table, src, dst, end, start=None, stream=None) -> None:
    """Copies positions between slots in every paged cache of a list at once (the layers' caches, which share one page
    table), on torch CUDA tensors: positions start[i] .. end[i]-1 of slot src[i] become those of slot dst[i]; -1 in either
    skips a row.  caches: [num_pages][2][Hk][page][d] tensors of one num_pages, page, d and element size; page_table:
    [num_slots][max_pages] int32; src, dst, end: [M] int32 on the device, start: [M] int32 or None (0).  No position that
    is written may be read or written by another row.  Without rows nothing is done.
    """
    array, n, device = _pools(caches)
    at = device.index
    like = caches[0]
    for c in caches:
        if c.dim() != 5 or c.shape[1] != 2 or c.shape[3:] != like.shape[3:] or c.element_size() != like.element_size():
            raise ValueError("every cache must be [num_pages][2][Hk][page][d] of the same page, d and element size")
    if page_table.dim() != 2 or not page_table.numel():
        raise ValueError("page_table must be [num_slots][max_pages]")
    num_slots, max_pages = shape = page_table.shape
    pages = _dense("page_table", page_table, shape, _torch().int32, at)
    M = int(src.shape[0])
    ids = _table32("src", src, M, at), _table32("dst", dst, M, at)
    first = 0 if start is None else _table32("start", start, M, at)
    last = _table32("end", end, M, at)
    if not M:
        return
    st = load().kda_pages_copy(ctypes.addressof(array), len(caches), n, like.shape[3], like.shape[4] * like.element_size(),
                               pages, num_slots, max_pages, *ids, first, last, M, _handle(stream, device))
    if st != KDA_OK:
        raise KdaError(st, "kda_pages_copy")


def beam_select(logits, scores, ended=None, end_token: int = -1, slots=None, stream=None):
    """One selection step of beam search, on torch CUDA tensors.

    logits: [G * B][V] bfloat16, float16 or float32, dense within a row, row g B + b for beam b of prompt g; scores: [G][B]
    float32, the beams' summed log probabilities (-inf: no hypothesis); ended: [G][B] int32 or None, with end_token: an
    ended beam stays as it is.  The best B of each prompt's candidates scores + log_softmax(logits), ties by the lowest
    beam and token.  slots: [G][B] int32 or None, the slots that hold the beams' states and caches.

    Returns (scores [G][B] float32, parents, tokens, ended, new_slots, src, dst), int32 [G][B]: each new beam's parent and
    token (-1 without a candidate), whether it has ended (None without an end_token), and, with slots, where its slot now
    is and which copies bring that about (src, dst for slots_copy and pages_copy, flattened; dst -1: none).
    """
    torch = _torch()
    at = _device_of("logits", logits)
    kinds = {torch.bfloat16: KDA_BF16, torch.float16: KDA_F16, torch.float32: KDA_F32}
    if logits.dtype not in kinds or logits.dim() != 2 or scores.dim() != 2:
        raise ValueError("logits must be [G * B][V] bfloat16, float16 or float32, scores [G][B]")
    rows, V = logits.shape
    G, B = shape = scores.shape
    if rows != G * B:
        raise ValueError("logits must have a row for each score")
    row, one = logits.stride()
    if one != 1 and V > 1:
        raise ValueError("logits must be dense within each row")
    s = _dense("scores", scores, shape, torch.float32, at)
    was = 0 if ended is None else _dense("ended", ended, shape, torch.int32, at)
    ids = 0 if slots is None else _dense("slots", slots, shape, torch.int32, at)
    device = logits.device
    stops, moves = end_token >= 0, slots is not None
    if not G:                                    # no prompt
        none = _new((7, 0, B), torch.int32, device, stream).unbind(0)
        return (none[0].view(torch.float32), *none[1:3], none[3] if stops else None) + (none[4:] if moves else (None,) * 3)
    lib = load()
    size = lib.kda_beam_select_workspace(G, B, V)
    if size <= 0:
        raise KdaError(KDA_ERR_SHAPE if B <= 64 and V <= 1 << 24 else KDA_ERR_UNSUPPORTED, "kda_beam_select")
    work = _scratch(size, device, stream)
    best, parents, tokens, stopped, new_slots, src, dst = _new((7, G, B), torch.int32, device, stream).unbind(0)
    best = best.view(torch.float32)              # one allocation for all
    st = lib.kda_beam_select(logits.data_ptr(), row if rows > 1 else V, kinds[logits.dtype], s, was, end_token, ids,
                             best.data_ptr(), parents.data_ptr(), tokens.data_ptr(), stopped.data_ptr() if stops else 0,
                             *((new_slots.data_ptr(), src.data_ptr(), dst.data_ptr()) if moves else (0, 0, 0)),
                             work.data_ptr(), size, G, B, V, _handle(stream, device))
    if st != KDA_OK:
        raise KdaError(st, "kda_beam_select")
    return (best, parents, tokens, stopped if stops else None) + ((new_slots, src, dst) if moves else (None, None, None))
