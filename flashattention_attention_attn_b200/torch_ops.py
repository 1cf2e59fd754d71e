"""torch custom ops over the C ABI, so that the kernels compose with
torch.compile (no graph break: the ops have fake/meta implementations that
give output shapes without running anything) and with CUDA-graph capture.

    import flashattention_attention_attn_b200.torch_ops  # registers the ops
    o, lse = torch.ops.fa_b200.attn_fwd(q, k, v, causal, scale)
    o, lse = torch.ops.fa_b200.attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, causal, scale)
    o, lse = torch.ops.fa_b200.paged_attn_prefill(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q,
                                                  max_seqlen_q, causal, scale)
    o = torch.ops.fa_b200.paged_attn_decode(q, k_cache, v_cache, block_table, seq_lens, num_splits)
    o = torch.ops.fa_b200.paged_attn_decode_fp8(q, k_cache, v_cache, block_table, seq_lens, num_splits,
                                                k_scale, v_scale)
    o_part, lse_part = torch.ops.fa_b200.paged_attn_decode_partial(q, k_cache, v_cache, block_table, seq_lens,
                                                                   num_splits)
    o = torch.ops.fa_b200.attn_lse_merge(o_parts, lse_parts)
    seq_lens, cu_seqlens_q, slot_map, positions, blocks_taken = torch.ops.fa_b200.paged_cache_plan(
        block_table, cached_lens, new_lens, free_blocks, pos_offsets, max_tokens)
    q, k = torch.ops.fa_b200.rope_axes(q, k, positions, inv_freq, freq_axis, adjacent)    # differentiable
    q = torch.ops.fa_b200.rope_axes_paged_append(q, k, v, positions, inv_freq, freq_axis, slot_map, adjacent,
                                                 k_cache, v_cache)
    q = torch.ops.fa_b200.rope_axes_paged_append_fp8(..., k_scale, v_scale)
    o, lse = torch.ops.fa_b200.paged_attn_prefill_fp8(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q,
                                                      max_seqlen_q, causal, scale, k_scale, v_scale, num_splits)

The op bodies only allocate the outputs and call the library on the current
stream; there is no other path.  Shapes follow include/attn.h:
q [B,T,Hq,d], k/v [B,S,Hkv,d] -> o [B,T,Hq,d], lse [B,Hq,T];
packed q [total_q,Hq,d], k/v [total_k,Hkv,d], cu_seqlens int32 [B+1]
-> o [total_q,Hq,d], lse [Hq,total_q];
decode q [B,Hq,d], caches [num_blocks,16,Hkv,d] (bf16, or e4m3 bytes),
block_table [B,max_blocks], seq_lens [B] -> o [B,Hq,d];
partial decode (the keys held here, the pool size read from the cache
shape) -> o_part [B,Hq,d] fp32, lse_part [B,Hq] fp32; merge of R partials
o_parts [R,B,Hq,d], lse_parts [R,B,Hq] -> o [B,Hq,d] bf16.
Plan: block_table [B,max_blocks] is updated in place, the other outputs are
new; pos_offsets may be None.  Rotary: q [n,Hq,d], k [n,Hkv,d] (rows of heads
may lie further apart, as columns of a fused projection do), positions
[axes,n] int32, inv_freq [rot/2] fp32, freq_axis a list of rot/2 axes (empty:
axis 0); the caches are written in place.  rope_axes has a gradient for q and
k, to the first order (rope_axes_bwd has none); an inv_freq that requires one is
refused.  It is captured into a graph under the rule of every torch operator: no
eager graph of the same leaves may live on the default stream meanwhile.
"""

from __future__ import annotations

import torch

from . import _binding


@torch.library.custom_op("fa_b200::attn_fwd", mutates_args=())
def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool,
             scale: float) -> tuple[torch.Tensor, torch.Tensor]:
    B, T, Hq, d = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    _binding.attn_fwd(q, k, v, o, lse, B, Hq, Hkv, T, S, d, causal, scale,
                      torch.cuda.current_stream(q.device))
    return o, lse


@attn_fwd.register_fake
def _(q, k, v, causal, scale):
    B, T, Hq, _ = q.shape
    return torch.empty_like(q), q.new_empty((B, Hq, T), dtype=torch.float32)


@torch.library.custom_op("fa_b200::paged_attn_decode", mutates_args=())
def paged_attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, num_splits: int) -> torch.Tensor:
    B, Hq, d = q.shape
    Hkv, block_size = k_cache.shape[2], k_cache.shape[1]
    o = torch.empty_like(q)
    _binding.paged_attn_decode(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size,
                               block_table.shape[1], num_splits, o, torch.cuda.current_stream(q.device))
    return o


@paged_attn_decode.register_fake
def _(q, k_cache, v_cache, block_table, seq_lens, num_splits):
    return torch.empty_like(q)


@torch.library.custom_op("fa_b200::attn_fwd_varlen", mutates_args=())
def attn_fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    cu_seqlens_k: torch.Tensor, max_seqlen_q: int, causal: bool,
                    scale: float) -> tuple[torch.Tensor, torch.Tensor]:
    total_q, Hq, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    B = cu_seqlens_q.shape[0] - 1
    o = torch.empty_like(q)
    lse = torch.empty((Hq, total_q), device=q.device, dtype=torch.float32)
    _binding.attn_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, max_seqlen_q, total_q, total_k, Hq,
                             Hkv, d, causal, scale, torch.cuda.current_stream(q.device))
    return o, lse


@attn_fwd_varlen.register_fake
def _(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, causal, scale):
    total_q, Hq, _ = q.shape
    return torch.empty_like(q), q.new_empty((Hq, total_q), dtype=torch.float32)


@torch.library.custom_op("fa_b200::paged_attn_prefill", mutates_args=())
def paged_attn_prefill(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, cu_seqlens_q: torch.Tensor, max_seqlen_q: int, causal: bool,
                       scale: float) -> tuple[torch.Tensor, torch.Tensor]:
    total_q, Hq, d = q.shape
    Hkv, block_size = k_cache.shape[2], k_cache.shape[1]
    B = cu_seqlens_q.shape[0] - 1
    o = torch.empty_like(q)
    lse = torch.empty((Hq, total_q), device=q.device, dtype=torch.float32)
    _binding.paged_attn_prefill(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, B, Hq, Hkv, d, block_size,
                                block_table.shape[1], max_seqlen_q, total_q, causal, scale, o, lse,
                                torch.cuda.current_stream(q.device))
    return o, lse


@paged_attn_prefill.register_fake
def _(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q, causal, scale):
    total_q, Hq, _ = q.shape
    return torch.empty_like(q), q.new_empty((Hq, total_q), dtype=torch.float32)


@torch.library.custom_op("fa_b200::paged_attn_decode_fp8", mutates_args=())
def paged_attn_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                          seq_lens: torch.Tensor, num_splits: int, k_scale: float, v_scale: float) -> torch.Tensor:
    B, Hq, d = q.shape
    Hkv, block_size = k_cache.shape[2], k_cache.shape[1]
    o = torch.empty_like(q)
    _binding.paged_attn_decode_fp8(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size,
                                   block_table.shape[1], num_splits, k_scale, v_scale, o,
                                   torch.cuda.current_stream(q.device))
    return o


@paged_attn_decode_fp8.register_fake
def _(q, k_cache, v_cache, block_table, seq_lens, num_splits, k_scale, v_scale):
    return torch.empty_like(q)


@torch.library.custom_op("fa_b200::paged_attn_decode_partial", mutates_args=())
def paged_attn_decode_partial(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              block_table: torch.Tensor, seq_lens: torch.Tensor,
                              num_splits: int) -> tuple[torch.Tensor, torch.Tensor]:
    B, Hq, d = q.shape
    num_blocks, block_size, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    o_part = torch.empty((B, Hq, d), device=q.device, dtype=torch.float32)
    lse_part = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
    if B > 0:  # the entry point takes no empty outputs
        _binding.paged_attn_decode_partial(q, k_cache, v_cache, block_table, seq_lens, B, Hq, Hkv, d, block_size,
                                           block_table.shape[1], num_blocks, num_splits, o_part, lse_part,
                                           torch.cuda.current_stream(q.device))
    return o_part, lse_part


@paged_attn_decode_partial.register_fake
def _(q, k_cache, v_cache, block_table, seq_lens, num_splits):
    B, Hq, _ = q.shape
    return q.new_empty(q.shape, dtype=torch.float32), q.new_empty((B, Hq), dtype=torch.float32)


@torch.library.custom_op("fa_b200::attn_lse_merge", mutates_args=())
def attn_lse_merge(o_parts: torch.Tensor, lse_parts: torch.Tensor) -> torch.Tensor:
    R, B, Hq, d = o_parts.shape
    o = torch.empty((B, Hq, d), device=o_parts.device, dtype=torch.bfloat16)
    if B > 0:
        _binding.attn_lse_merge(o_parts, lse_parts, R, B, Hq, d, o, torch.cuda.current_stream(o_parts.device))
    return o


@attn_lse_merge.register_fake
def _(o_parts, lse_parts):
    return o_parts.new_empty(o_parts.shape[1:], dtype=torch.bfloat16)


def _packed(x: torch.Tensor) -> torch.Tensor:
    """x without gaps and on a 16-byte boundary, copied only if it is not (a slice of a flat buffer may be packed and
    lie off the boundary, where contiguous() copies nothing)."""
    return x.contiguous() if not x.is_contiguous() or x.data_ptr() % 16 == 0 else x.clone()


def _rows(x: torch.Tensor) -> torch.Tensor:
    """x [n, H, d] with the heads of a row side by side and the rows apart, copied only if they are not
    (a gradient that was expanded over the tokens has rows that share their memory)."""
    if (x.stride(-1) != 1 or (x.shape[1] > 1 and x.stride(1) != x.shape[2]) or x.stride(0) % 8 or x.data_ptr() % 16
            or (x.shape[0] > 1 and x.stride(0) < x.shape[1] * x.shape[2])):
        return _packed(x)
    return x


_BF16, _INT32, _FP32 = (torch.bfloat16,), (torch.int32,), (torch.float32,)
_FP8 = (torch.uint8, torch.float8_e4m3fn)


def _need(packed: bool, dtypes, **tensors) -> None:
    """The types that the entry points read behind their pointers and, packed, no gaps."""
    for name, x in tensors.items():
        if x is None:
            continue
        if x.dtype not in dtypes:
            raise ValueError(f"{name} is {x.dtype}, not {' or '.join(str(t) for t in dtypes)}")
        if packed and not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _shape(**tensors) -> None:
    """name=(tensor, shape): the sizes that the entry points take from the other tensors; None stands for any."""
    for name, (x, want) in tensors.items():
        if x is not None and (x.dim() != len(want) or any(w is not None and n != w for n, w in zip(x.shape, want))):
            raise ValueError(f"{name} is {tuple(x.shape)}, not {tuple('any' if w is None else w for w in want)}")


def _stride(x: torch.Tensor) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1] * x.shape[2]


def _positions(positions: torch.Tensor) -> torch.Tensor:
    return positions if positions.stride(-1) == 1 or positions.shape[-1] == 1 else positions.contiguous()


@torch.library.custom_op("fa_b200::paged_cache_plan", mutates_args=("block_table",))
def paged_cache_plan(block_table: torch.Tensor, cached_lens: torch.Tensor, new_lens: torch.Tensor,
                     free_blocks: torch.Tensor, pos_offsets: torch.Tensor | None, max_tokens: int
                     ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    _need(True, _INT32, block_table=block_table, cached_lens=cached_lens, new_lens=new_lens, free_blocks=free_blocks,
          pos_offsets=pos_offsets)
    _shape(block_table=(block_table, (None, None)), free_blocks=(free_blocks, (None,)))
    B, max_blocks = block_table.shape
    _shape(cached_lens=(cached_lens, (B,)), new_lens=(new_lens, (B,)), pos_offsets=(pos_offsets, (B,)))
    out = [torch.empty(n, device=block_table.device, dtype=torch.int32)
           for n in (B, B + 1, max_tokens, max_tokens, 1)]
    seq_lens, cu, slots, positions, taken = out
    with torch.cuda.device(block_table.device):  # the call is made on, and its stream taken from, the tensors' device
        _binding.paged_cache_plan(cached_lens, new_lens, free_blocks, pos_offsets, B, free_blocks.numel(), 16, max_blocks,
                                  max_tokens, block_table, seq_lens, cu, slots, positions, taken)
    return seq_lens, cu, slots, positions, taken


@paged_cache_plan.register_fake
def _(block_table, cached_lens, new_lens, free_blocks, pos_offsets, max_tokens):
    B = block_table.shape[0]
    return tuple(block_table.new_empty(n, dtype=torch.int32) for n in (B, B + 1, max_tokens, max_tokens, 1))


def _rope(call, q, k, positions, inv_freq, freq_axis, adjacent):
    _need(False, _BF16, q=q, k=k)
    _need(False, _INT32, positions=positions)
    _need(True, _FP32, inv_freq=inv_freq)
    _shape(q=(q, (None, None, None)))
    n, Hq, d = q.shape
    _shape(k=(k, (n, None, d)), positions=(positions, (None, n)), inv_freq=(inv_freq, (None,)))
    Hkv = k.shape[1]
    q, k, positions = _rows(q), _rows(k), _positions(positions)
    q_out = torch.empty((n, Hq, d), device=q.device, dtype=q.dtype)
    k_out = torch.empty((n, Hkv, d), device=q.device, dtype=q.dtype)
    with torch.cuda.device(q.device):
        call(q, k, positions, inv_freq, freq_axis or None, n, Hq, Hkv, d, 2 * inv_freq.numel(), positions.shape[0],
             positions.stride(0), _stride(q), _stride(k), adjacent, q_out, k_out, Hq * d, Hkv * d)
    return q_out, k_out


def _rope_fake(q, k, positions, inv_freq, freq_axis, adjacent):
    return q.new_empty(q.shape), k.new_empty(k.shape)


@torch.library.custom_op("fa_b200::rope_axes", mutates_args=())
def rope_axes(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, freq_axis: list[int],
              adjacent: bool) -> tuple[torch.Tensor, torch.Tensor]:
    return _rope(_binding.rope_axes_fwd, q, k, positions, inv_freq, freq_axis, adjacent)


@torch.library.custom_op("fa_b200::rope_axes_bwd", mutates_args=())
def rope_axes_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                  freq_axis: list[int], adjacent: bool) -> tuple[torch.Tensor, torch.Tensor]:
    return _rope(_binding.rope_axes_bwd, dq_out, dk_out, positions, inv_freq, freq_axis, adjacent)


rope_axes.register_fake(_rope_fake)
rope_axes_bwd.register_fake(_rope_fake)


def _rope_setup(ctx, inputs, output):
    _, _, positions, inv_freq, ctx.freq_axis, ctx.adjacent = inputs
    if ctx.needs_input_grad[3]:
        raise ValueError("inv_freq requires a gradient, which rope_axes does not compute: pass inv_freq.detach()")
    ctx.save_for_backward(positions, inv_freq)


def _rope_backward(ctx, dq_out, dk_out):
    positions, inv_freq = ctx.saved_tensors
    dq, dk = torch.ops.fa_b200.rope_axes_bwd(dq_out, dk_out, positions, inv_freq, ctx.freq_axis, ctx.adjacent)
    return dq, dk, None, None, None, None


rope_axes.register_autograd(_rope_backward, setup_context=_rope_setup)


def _append(q, k, v, positions, inv_freq, freq_axis, slot_map, adjacent, k_cache, v_cache, scales):
    _need(False, _BF16, q=q, k=k, v=v)
    _need(False, _INT32, positions=positions)
    _need(True, _INT32, slot_map=slot_map)
    _need(True, _FP32, inv_freq=inv_freq)
    _need(True, _FP8 if scales else _BF16, k_cache=k_cache, v_cache=v_cache)
    _shape(q=(q, (None, None, None)), k_cache=(k_cache, (None, None, None, None)))
    n, Hq, d = q.shape
    num_blocks, block_size, Hkv = k_cache.shape[:3]
    _shape(k=(k, (n, Hkv, d)), v=(v, (n, Hkv, d)), positions=(positions, (None, n)), inv_freq=(inv_freq, (None,)),
           slot_map=(slot_map, (n,)), k_cache=(k_cache, (num_blocks, block_size, Hkv, d)),
           v_cache=(v_cache, (num_blocks, block_size, Hkv, d)))
    q, k, v, positions = _rows(q), _rows(k), _rows(v), _positions(positions)
    q_out = torch.empty((n, Hq, d), device=q.device, dtype=q.dtype)
    call = _binding.rope_axes_paged_append_fp8 if scales else _binding.rope_axes_paged_append
    with torch.cuda.device(q.device):
        call(q, k, v, positions, inv_freq, freq_axis or None, slot_map, n, Hq, Hkv, d, 2 * inv_freq.numel(),
             positions.shape[0], positions.stride(0), _stride(q), _stride(k), _stride(v), adjacent, block_size,
             num_blocks, *scales, q_out, k_cache, v_cache)
    return q_out


@torch.library.custom_op("fa_b200::rope_axes_paged_append", mutates_args=("k_cache", "v_cache"))
def rope_axes_paged_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                           inv_freq: torch.Tensor, freq_axis: list[int], slot_map: torch.Tensor, adjacent: bool,
                           k_cache: torch.Tensor, v_cache: torch.Tensor) -> torch.Tensor:
    return _append(q, k, v, positions, inv_freq, freq_axis, slot_map, adjacent, k_cache, v_cache, ())


@rope_axes_paged_append.register_fake
def _(q, k, v, positions, inv_freq, freq_axis, slot_map, adjacent, k_cache, v_cache):
    return q.new_empty(q.shape)


@torch.library.custom_op("fa_b200::rope_axes_paged_append_fp8", mutates_args=("k_cache", "v_cache"))
def rope_axes_paged_append_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                               inv_freq: torch.Tensor, freq_axis: list[int], slot_map: torch.Tensor, adjacent: bool,
                               k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float,
                               v_scale: float) -> torch.Tensor:
    return _append(q, k, v, positions, inv_freq, freq_axis, slot_map, adjacent, k_cache, v_cache, (k_scale, v_scale))


@rope_axes_paged_append_fp8.register_fake
def _(q, k, v, positions, inv_freq, freq_axis, slot_map, adjacent, k_cache, v_cache, k_scale, v_scale):
    return q.new_empty(q.shape)


@torch.library.custom_op("fa_b200::paged_attn_prefill_fp8", mutates_args=())
def paged_attn_prefill_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                           seq_lens: torch.Tensor, cu_seqlens_q: torch.Tensor, max_seqlen_q: int, causal: bool,
                           scale: float, k_scale: float, v_scale: float,
                           num_splits: int) -> tuple[torch.Tensor, torch.Tensor]:
    _need(False, _BF16, q=q)
    _need(True, _FP8, k_cache=k_cache, v_cache=v_cache)
    _need(True, _INT32, block_table=block_table, seq_lens=seq_lens, cu_seqlens_q=cu_seqlens_q)
    _shape(q=(q, (None, None, None)), k_cache=(k_cache, (None, None, None, None)),
           cu_seqlens_q=(cu_seqlens_q, (None,)))
    q = _packed(q)
    total_q, Hq, d = q.shape
    num_blocks, block_size, Hkv = k_cache.shape[:3]
    B = cu_seqlens_q.shape[0] - 1
    _shape(k_cache=(k_cache, (num_blocks, block_size, Hkv, d)), v_cache=(v_cache, (num_blocks, block_size, Hkv, d)),
           block_table=(block_table, (B, None)), seq_lens=(seq_lens, (B,)))
    o = torch.empty((total_q, Hq, d), device=q.device, dtype=q.dtype)
    lse = torch.empty((Hq, total_q), device=q.device, dtype=torch.float32)
    if B > 0:
        with torch.cuda.device(q.device):
            _binding.paged_attn_prefill_fp8_checked(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, B, Hq, Hkv,
                                                    d, block_size, block_table.shape[1], num_blocks, max_seqlen_q,
                                                    total_q, causal, scale, k_scale, v_scale, num_splits, o, lse)
    return o, lse


@paged_attn_prefill_fp8.register_fake
def _(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q, causal, scale, k_scale, v_scale,
      num_splits):
    total_q, Hq, _ = q.shape
    return q.new_empty(q.shape), q.new_empty((Hq, total_q), dtype=torch.float32)
