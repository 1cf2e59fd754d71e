"""ctypes binding of the C ABI in include/attn.h.

Argument marshalling only: tensors become device pointers, the current
torch stream becomes the cudaStream_t, and a non-zero status becomes an
exception.  Every step of the computation runs in the CUDA library; if it
cannot be loaded, every call raises.
"""

from __future__ import annotations

import ctypes
import os

import torch

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libattn_b200.so")

ATTN_OK = 0
ATTN_DEVSTATUS_TIMEOUT = 0x1
ATTN_DEVSTATUS_BAD_BLOCK = 0x2
ATTN_DEVSTATUS_BAD_SEQLEN = 0x4
ATTN_DEVSTATUS_NO_BLOCK = 0x8
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {attn_status_string(status)} (status {status})")


def library() -> ctypes.CDLL:
    """Load the library once (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"CUDA library not built: {library_path} is missing "
                "(run `python -m flashattention_attention_attn_b200.build`)")
        lib = ctypes.CDLL(library_path)
        c_int, c_float, vp = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
        lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_float, vp]
        lib.attn_fwd.restype = c_int
        lib.attn_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                        c_int, c_float, vp]
        lib.attn_fwd_varlen.restype = c_int
        lib.paged_attn_prefill.argtypes = [vp, vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                           c_int, c_int, c_float, vp, vp, vp]
        lib.paged_attn_prefill.restype = c_int
        lib.paged_attn_decode.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                          vp, vp]
        lib.paged_attn_decode.restype = c_int
        lib.paged_attn_decode_fp8.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                              c_float, c_float, vp, vp]
        lib.paged_attn_decode_fp8.restype = c_int
        lib.paged_attn_decode_noalloc.argtypes = lib.paged_attn_decode.argtypes
        lib.paged_attn_decode_noalloc.restype = c_int
        lib.paged_attn_decode_checked.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int,
                                                  c_int, c_int, vp, vp]
        lib.paged_attn_decode_checked.restype = c_int
        lib.paged_attn_decode_fp8_checked.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int,
                                                      c_int, c_int, c_float, c_float, vp, vp]
        lib.paged_attn_decode_fp8_checked.restype = c_int
        lib.paged_attn_prefill_checked.argtypes = [vp, vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int,
                                                   c_int, c_int, c_int, c_int, c_float, vp, vp, vp]
        lib.paged_attn_prefill_checked.restype = c_int
        lib.paged_attn_decode_partial.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int,
                                                  c_int, c_int, vp, vp, vp]
        lib.paged_attn_decode_partial.restype = c_int
        lib.attn_lse_merge.argtypes = [vp, vp, c_int, c_int, c_int, c_int, vp, vp]
        lib.attn_lse_merge.restype = c_int
        i64, c_bytes = ctypes.c_int64, ctypes.c_char_p
        lib.paged_cache_plan.argtypes = [vp] * 4 + [c_int] * 5 + [vp] * 7
        lib.paged_cache_plan.restype = c_int
        rope_head = [vp, vp, vp, vp, c_bytes]
        lib.rope_axes_fwd.argtypes = rope_head + [c_int] * 6 + [i64] * 3 + [c_int, vp, vp, i64, i64, vp]
        lib.rope_axes_fwd.restype = c_int
        lib.rope_axes_bwd.argtypes = lib.rope_axes_fwd.argtypes
        lib.rope_axes_bwd.restype = c_int
        append_head = [vp] * 5 + [c_bytes, vp] + [c_int] * 6 + [i64] * 4 + [c_int] * 3
        lib.rope_axes_paged_append.argtypes = append_head + [vp] * 4
        lib.rope_axes_paged_append.restype = c_int
        lib.rope_axes_paged_append_fp8.argtypes = append_head + [c_float] * 2 + [vp] * 4
        lib.rope_axes_paged_append_fp8.restype = c_int
        lib.paged_attn_prefill_fp8.argtypes = [vp] * 6 + [c_int] * 9 + [c_float] * 3 + [c_int] + [vp] * 3
        lib.paged_attn_prefill_fp8.restype = c_int
        lib.paged_attn_prefill_fp8_checked.argtypes = [vp] * 6 + [c_int] * 10 + [c_float] * 3 + [c_int] + [vp] * 3
        lib.paged_attn_prefill_fp8_checked.restype = c_int
        lib.attn_check_support.argtypes = [c_int]
        lib.attn_check_support.restype = c_int
        lib.attn_status_string.argtypes = [c_int]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_read_device_status.argtypes = [ctypes.POINTER(c_int), c_int]
        lib.attn_read_device_status.restype = c_int
        lib.attn_selftest_bounded_wait.argtypes = [vp]
        lib.attn_selftest_bounded_wait.restype = c_int
        _lib = lib
    return _lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr() if x.numel() > 0 else None
    return int(x)


def _pointers(*xs):
    """Device pointers for a call on the current device; a tensor that lives
    elsewhere (another GPU, the host) is refused."""
    dev = torch.cuda.current_device()
    out = []
    for x in xs:
        if isinstance(x, torch.Tensor):
            if x.get_device() != dev:
                raise ValueError(f"a tensor on {x.device} in a call on cuda:{dev} (the current device)")
            x = x.data_ptr() or None
        out.append(x)
    return out


def _stream(stream) -> int | None:
    if stream is None:  # the handle alone: a torch.cuda.Stream object costs 3 us a call, this 0.3
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def attn_status_string(status: int) -> str:
    return library().attn_status_string(int(status)).decode()


def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, T, S, d, causal, scale, stream=None) -> None:
    """O = softmax(scale * Q K^T [+ causal mask]) V, plus LSE.

    q [B,T,Hq,d], k/v [B,S,Hkv,d], o [B,T,Hq,d] bf16; lse [B,Hq,T] fp32 or None.
    """
    rc = library().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq), int(Hkv), int(T),
                            int(S), int(d), int(bool(causal)), float(scale), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd")


def attn_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, max_seqlen_q, total_q, total_k, Hq, Hkv, d,
                    causal, scale, stream=None) -> None:
    """attn_fwd over packed sequences: q [total_q,Hq,d], k/v [total_k,Hkv,d],
    o [total_q,Hq,d], lse [Hq,total_q] or None, cu_seqlens_* int32 [B+1]."""
    rc = library().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q),
                                   _ptr(cu_seqlens_k), int(B), int(max_seqlen_q), int(total_q), int(total_k),
                                   int(Hq), int(Hkv), int(d), int(bool(causal)), float(scale), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_varlen")


def paged_attn_prefill(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, B, Hq, Hkv, d, block_size,
                       max_blocks, max_seqlen_q, total_q, causal, scale, o, lse, stream=None) -> None:
    """Chunked prefill against the paged cache (see attn.h)."""
    rc = library().paged_attn_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                      _ptr(cu_seqlens_q), int(B), int(Hq), int(Hkv), int(d), int(block_size),
                                      int(max_blocks), int(max_seqlen_q), int(total_q), int(bool(causal)),
                                      float(scale), _ptr(o), _ptr(lse), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_prefill")


def paged_attn_decode(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size, max_blocks,
                      num_splits, o, stream=None) -> None:
    """One query token per sequence against a paged KV cache (see attn.h)."""
    rc = library().paged_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                     int(B), int(Hq), int(Hkv), int(d), int(block_size), int(max_blocks),
                                     int(num_splits), _ptr(o), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_decode")


def paged_attn_decode_fp8(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size, max_blocks,
                          num_splits, k_scale, v_scale, o, stream=None) -> None:
    """paged_attn_decode over an FP8 e4m3 cache with per-tensor scales (see attn.h)."""
    rc = library().paged_attn_decode_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                         int(B), int(Hq), int(Hkv), int(d), int(block_size), int(max_blocks),
                                         int(num_splits), float(k_scale), float(v_scale), _ptr(o), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_decode_fp8")


def paged_attn_decode_checked(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size, max_blocks,
                              num_blocks, num_splits, o, stream=None) -> None:
    """paged_attn_decode for a pool of num_blocks blocks: table entries
    outside it are masked and flagged (see attn.h)."""
    rc = library().paged_attn_decode_checked(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                             _ptr(seq_lens), int(B), int(Hq), int(Hkv), int(d), int(block_size),
                                             int(max_blocks), int(num_blocks), int(num_splits), _ptr(o),
                                             _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_decode_checked")


def paged_attn_decode_partial(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size, max_blocks,
                              num_blocks, num_splits, o_part, lse_part, stream=None) -> None:
    """Decode over the keys held here, as fp32 o_part [B, Hq, d] and
    lse_part [B, Hq] for a later attn_lse_merge (see attn.h)."""
    rc = library().paged_attn_decode_partial(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                             _ptr(seq_lens), int(B), int(Hq), int(Hkv), int(d), int(block_size),
                                             int(max_blocks), int(num_blocks), int(num_splits), _ptr(o_part),
                                             _ptr(lse_part), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_decode_partial")


def attn_lse_merge(o_parts, lse_parts, R, B, Hq, d, o, stream=None) -> None:
    """Merge R partial results [R, B, Hq, d] / [R, B, Hq] into bf16 o [B, Hq, d] (see attn.h)."""
    rc = library().attn_lse_merge(_ptr(o_parts), _ptr(lse_parts), int(R), int(B), int(Hq), int(d), _ptr(o),
                                  _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_lse_merge")


def paged_attn_decode_fp8_checked(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size, max_blocks,
                                  num_blocks, num_splits, k_scale, v_scale, o, stream=None) -> None:
    """paged_attn_decode_fp8 for a pool of num_blocks blocks (see attn.h)."""
    rc = library().paged_attn_decode_fp8_checked(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                                 _ptr(seq_lens), int(B), int(Hq), int(Hkv), int(d), int(block_size),
                                                 int(max_blocks), int(num_blocks), int(num_splits), float(k_scale),
                                                 float(v_scale), _ptr(o), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_decode_fp8_checked")


def paged_attn_prefill_checked(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, B, Hq, Hkv, d, block_size,
                               max_blocks, num_blocks, max_seqlen_q, total_q, causal, scale, o, lse,
                               stream=None) -> None:
    """paged_attn_prefill for a pool of num_blocks blocks (see attn.h)."""
    rc = library().paged_attn_prefill_checked(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                              _ptr(seq_lens), _ptr(cu_seqlens_q), int(B), int(Hq), int(Hkv), int(d),
                                              int(block_size), int(max_blocks), int(num_blocks), int(max_seqlen_q),
                                              int(total_q), int(bool(causal)), float(scale), _ptr(o), _ptr(lse),
                                              _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_prefill_checked")


def paged_attn_decode_noalloc(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size,
                              max_blocks, num_splits, o, stream=None) -> None:
    """paged_attn_decode with its split partials in the library's fixed
    scratch array: for callers that must not allocate during the call (see
    attn.h for the size limit and the sharing rules)."""
    rc = library().paged_attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                             _ptr(seq_lens), int(B), int(Hq), int(Hkv), int(d), int(block_size),
                                             int(max_blocks), int(num_splits), _ptr(o), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_decode_noalloc")


def paged_cache_plan(cached_lens, new_lens, free_blocks, pos_offsets, B, num_free, block_size, max_blocks, max_tokens,
                     block_table, seq_lens, cu_seqlens_q, slot_map, positions, blocks_taken, stream=None) -> None:
    """Block-table entries, slots, positions and prefix sums of a step's new
    tokens from the requests' lengths (see attn.h)."""
    ins = _pointers(cached_lens, new_lens, free_blocks, pos_offsets)
    outs = _pointers(block_table, seq_lens, cu_seqlens_q, slot_map, positions, blocks_taken)
    rc = library().paged_cache_plan(*ins, int(B), int(num_free), int(block_size), int(max_blocks), int(max_tokens), *outs,
                                    _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_cache_plan")


def rope_axis_map(sections, interleaved=False) -> bytes:
    """freq_axis of the rotary calls: sections[a] pairs rotate with axis a.

    In contiguous runs (the first sections[0] pairs with axis 0, and so on),
    or, interleaved, dealt out in turn (axis 0, 1, .., 0, 1, ..) until a
    section is used up.
    """
    left = [int(n) for n in sections]
    if any(n < 0 for n in left) or len(left) > 255:
        raise ValueError("sections: up to 255 counts of pairs, none negative")
    if not interleaved:
        return b"".join(bytes([a]) * n for a, n in enumerate(left))
    out = bytearray()
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] = n - 1
    return bytes(out)


def _axis_bytes(freq_axis, rot_dim) -> bytes | None:
    if freq_axis is None:
        return None
    axes = bytes(freq_axis)
    if len(axes) != int(rot_dim) // 2:
        raise ValueError(f"freq_axis has {len(axes)} entries, rot_dim {rot_dim} needs {int(rot_dim) // 2}")
    return axes


def _rope(name, q, k, positions, inv_freq, freq_axis, n_tokens, Hq, Hkv, d, rot_dim, num_axes, pos_stride, q_stride,
          k_stride, adjacent, q_out, k_out, q_out_stride, k_out_stride, stream) -> None:
    axes = _axis_bytes(freq_axis, rot_dim)
    q, k, positions, inv_freq, q_out, k_out = _pointers(q, k, positions, inv_freq, q_out, k_out)
    rc = getattr(library(), name)(q, k, positions, inv_freq, axes, int(n_tokens), int(Hq), int(Hkv), int(d), int(rot_dim),
                                  int(num_axes), int(pos_stride), int(q_stride), int(k_stride), int(bool(adjacent)),
                                  q_out, k_out, int(q_out_stride), int(k_out_stride), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, name)


def rope_axes_fwd(q, k, positions, inv_freq, freq_axis, n_tokens, Hq, Hkv, d, rot_dim, num_axes, pos_stride, q_stride,
                  k_stride, adjacent, q_out, k_out, q_out_stride, k_out_stride, stream=None) -> None:
    """Rotary positions with several axes (see attn.h).  freq_axis: bytes or
    ints, the axis of each of the rot_dim / 2 pairs (rope_axis_map), or None."""
    _rope("rope_axes_fwd", q, k, positions, inv_freq, freq_axis, n_tokens, Hq, Hkv, d, rot_dim, num_axes, pos_stride,
          q_stride, k_stride, adjacent, q_out, k_out, q_out_stride, k_out_stride, stream)


def rope_axes_bwd(dq_out, dk_out, positions, inv_freq, freq_axis, n_tokens, Hq, Hkv, d, rot_dim, num_axes, pos_stride,
                  dq_out_stride, dk_out_stride, adjacent, dq, dk, dq_stride, dk_stride, stream=None) -> None:
    """Gradient of rope_axes_fwd (see attn.h)."""
    _rope("rope_axes_bwd", dq_out, dk_out, positions, inv_freq, freq_axis, n_tokens, Hq, Hkv, d, rot_dim, num_axes,
          pos_stride, dq_out_stride, dk_out_stride, adjacent, dq, dk, dq_stride, dk_stride, stream)


def _rope_append(name, q, k, v, positions, inv_freq, freq_axis, slot_map, n_tokens, Hq, Hkv, d, rot_dim, num_axes,
                 pos_stride, q_stride, k_stride, v_stride, adjacent, block_size, num_blocks, scales, q_out, k_cache,
                 v_cache, stream) -> None:
    axes = _axis_bytes(freq_axis, rot_dim)
    q, k, v, positions, inv_freq, slot_map, q_out, k_cache, v_cache = _pointers(
        q, k, v, positions, inv_freq, slot_map, q_out, k_cache, v_cache)
    rc = getattr(library(), name)(q, k, v, positions, inv_freq, axes, slot_map, int(n_tokens), int(Hq), int(Hkv), int(d),
                                  int(rot_dim), int(num_axes), int(pos_stride), int(q_stride), int(k_stride),
                                  int(v_stride), int(bool(adjacent)), int(block_size), int(num_blocks), *scales, q_out,
                                  k_cache, v_cache, _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, name)


def rope_axes_paged_append(q, k, v, positions, inv_freq, freq_axis, slot_map, n_tokens, Hq, Hkv, d, rot_dim, num_axes,
                           pos_stride, q_stride, k_stride, v_stride, adjacent, block_size, num_blocks, q_out, k_cache,
                           v_cache, stream=None) -> None:
    """rope_axes_fwd of q and k, with k and v written into the paged bf16
    cache at slot_map (see attn.h)."""
    _rope_append("rope_axes_paged_append", q, k, v, positions, inv_freq, freq_axis, slot_map, n_tokens, Hq, Hkv, d,
                 rot_dim, num_axes, pos_stride, q_stride, k_stride, v_stride, adjacent, block_size, num_blocks, (), q_out,
                 k_cache, v_cache, stream)


def rope_axes_paged_append_fp8(q, k, v, positions, inv_freq, freq_axis, slot_map, n_tokens, Hq, Hkv, d, rot_dim,
                               num_axes, pos_stride, q_stride, k_stride, v_stride, adjacent, block_size, num_blocks,
                               k_scale, v_scale, q_out, k_cache, v_cache, stream=None) -> None:
    """rope_axes_paged_append into an FP8 e4m3 cache with per-tensor scales (see attn.h)."""
    _rope_append("rope_axes_paged_append_fp8", q, k, v, positions, inv_freq, freq_axis, slot_map, n_tokens, Hq, Hkv, d,
                 rot_dim, num_axes, pos_stride, q_stride, k_stride, v_stride, adjacent, block_size, num_blocks,
                 (float(k_scale), float(v_scale)), q_out, k_cache, v_cache, stream)


def paged_attn_prefill_fp8(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, B, Hq, Hkv, d, block_size,
                           max_blocks, max_seqlen_q, total_q, causal, scale, k_scale, v_scale, num_splits, o, lse,
                           stream=None) -> None:
    """Chunked prefill against an FP8 e4m3 paged cache with per-tensor scales (see attn.h)."""
    ptrs = _pointers(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, o, lse)
    rc = library().paged_attn_prefill_fp8(*ptrs[:6], int(B), int(Hq), int(Hkv), int(d), int(block_size), int(max_blocks),
                                          int(max_seqlen_q), int(total_q), int(bool(causal)), float(scale),
                                          float(k_scale), float(v_scale), int(num_splits), *ptrs[6:], _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_prefill_fp8")


def paged_attn_prefill_fp8_checked(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, B, Hq, Hkv, d, block_size,
                                   max_blocks, num_blocks, max_seqlen_q, total_q, causal, scale, k_scale, v_scale,
                                   num_splits, o, lse, stream=None) -> None:
    """paged_attn_prefill_fp8 for a pool of num_blocks blocks (see attn.h)."""
    ptrs = _pointers(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, o, lse)
    rc = library().paged_attn_prefill_fp8_checked(*ptrs[:6], int(B), int(Hq), int(Hkv), int(d), int(block_size),
                                                  int(max_blocks), int(num_blocks), int(max_seqlen_q), int(total_q),
                                                  int(bool(causal)), float(scale), float(k_scale), float(v_scale),
                                                  int(num_splits), *ptrs[6:], _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "paged_attn_prefill_fp8_checked")


def attn_check_support(device: int = 0) -> int:
    return int(library().attn_check_support(int(device)))


def attn_read_device_status(clear: bool = True) -> int:
    out = ctypes.c_int(0)
    rc = library().attn_read_device_status(ctypes.byref(out), int(bool(clear)))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_read_device_status")
    return int(out.value)


def attn_selftest_bounded_wait(stream=None) -> None:
    """Launch the bounded-wait self test (see attn.h); read the outcome with
    attn_read_device_status()."""
    rc = library().attn_selftest_bounded_wait(_stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_selftest_bounded_wait")
