"""The serving step around the paged cache, operator by operator: inputs, plain form, 64-bit form and work of each case.

Four operators that follow one another in a step of a server (and the rotary one in a training step as well):

  plan    paged_cache_plan: block tables, slot map, positions and prefix sums from the requests' lengths
  rope    rope_axes_fwd / rope_axes_bwd: rotary positions with several axes, and the gradient
  append  rope_axes_paged_append(_fp8): the same rotation of q and k, with k and v written into the paged cache
  chunk   paged_attn_prefill_fp8_checked: attention of each sequence's new tokens over its FP8 (e4m3) paged cache

A case's lengths come from its own "lens" number, so that its work is known without its inputs; every other value comes
from the seed.  `run` computes the plain form in torch operations when `own` is false, and calls the library when it
is true.
"""

from __future__ import annotations

import math
import random

import torch

own = False

BS = 16  # tokens per cache block
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
ROPE_BASE = 500000.0


def listed():
    return [
        # one new token for each of 64 running requests: the plan of a decode step, where latency is all
        dict(name="plan_decode_b64", op="plan", B=64, c_lo=256, c_hi=4096, n_lo=1, n_hi=1, max_blocks=257, pad=0, lens=1),
        # a large pool of requests, from finished ones (no new token) to 64-token chunks, in a batch padded for a graph
        dict(name="plan_ragged_b4096", op="plan", B=4096, c_lo=0, c_hi=4000, n_lo=0, n_hi=64, max_blocks=256, pad=1000,
             lens=2),
        # the rotation of a training step over 16k image, video and text tokens (time, height, width axes)
        dict(name="rope_fwd_16k", op="rope", dir="fwd", n=16384, Hq=32, Hkv=8, d=128, rot=128, axes=3, pairs="half",
             fused=True),
        # the gradient of an odd-sized batch, heads of 64 with half of each rotated, adjacent pairs
        dict(name="rope_bwd_4099_d64", op="rope", dir="bwd", n=4099, Hq=16, Hkv=16, d=64, rot=32, axes=2, pairs="adjacent",
             fused=False),
        # the cache write of a decode step: 64 tokens, one for each sequence
        dict(name="append_decode_b64", op="append", cache="bf16", B=64, c_lo=256, c_hi=4096, n_lo=1, n_hi=1, Hq=32, Hkv=8,
             d=128, rot=128, axes=1, pairs="half", lens=3),
        # eight 512-token chunks of image and text tokens into an FP8 cache
        dict(name="append_fp8_8x512", op="append", cache="fp8", B=8, c_lo=512, c_hi=7680, n_lo=512, n_hi=512, Hq=32, Hkv=8,
             d=128, rot=128, axes=3, pairs="half", lens=4),
        # ragged prompts of up to 2k tokens, heads of 64, adjacent pairs
        dict(name="append_ragged_d64", op="append", cache="bf16", B=16, c_lo=0, c_hi=0, n_lo=64, n_hi=2048, Hq=24, Hkv=4,
             d=64, rot=64, axes=2, pairs="adjacent", lens=5),
        # four drafted tokens of each of 64 requests checked in one pass: few rows, bound by the cache's bytes
        dict(name="chunk_verify_b64x4", op="chunk", B=64, c_lo=252, c_hi=4092, n_lo=4, n_hi=4, Hq=32, Hkv=8, causal=True,
             lens=6),
        # running requests and new prompts in one batch: no new token, a few, or hundreds; six query heads share a kv head
        dict(name="chunk_ragged_b33_g6", op="chunk", B=33, c_lo=0, c_hi=2500, n_lo=0, n_hi=300, Hq=24, Hkv=4, causal=True,
             lens=7),
        # the chunked prefill of eight requests with 1k to 8k tokens behind them
        dict(name="chunk_8x512", op="chunk", B=8, c_lo=512, c_hi=7680, n_lo=512, n_hi=512, Hq=32, Hkv=8, causal=True,
             lens=8),
        # a question of eight tokens about a 131k-token document: one long axis, few rows, every key seen
        dict(name="chunk_long_131k_x8", op="chunk", B=1, c_lo=131064, c_hi=131064, n_lo=8, n_hi=8, Hq=32, Hkv=8,
             causal=False, lens=9),
        # a 2k-token chunk late in a long prompt: bound by the tensor cores
        dict(name="chunk_2048_at_32k", op="chunk", B=1, c_lo=30720, c_hi=30720, n_lo=2048, n_hi=2048, Hq=32, Hkv=8,
             causal=True, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "chunk", "chunk"])
    lens = rng.randrange(1, 1 << 30)
    if op == "plan":
        B = _log(rng, 1, 4096)
        n_hi = _log(rng, 1, max(1, min(2048, 131072 // B)))
        c_hi = _log(rng, 1, 4000)
        return dict(op=op, B=B, c_lo=0, c_hi=c_hi, n_lo=rng.choice([0, 1]), n_hi=n_hi, max_blocks=(c_hi + n_hi) // BS + 1,
                    pad=rng.choice([0, 0, rng.randrange(1, 500)]), lens=lens)
    d = rng.choice([64, 128])
    G, Hkv = rng.choice([(1, 8), (2, 4), (3, 2), (4, 8), (4, 1), (5, 8), (6, 4), (7, 4), (8, 4), (8, 8)])
    if op == "rope":
        n = _log(rng, 1, 16384 * 40 // (Hkv * (G + 1)))
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), n=min(n, 65536), Hq=G * Hkv, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d, d // 2]), axes=rng.choice([1, 2, 3]), pairs=rng.choice(["half", "adjacent"]),
                    fused=rng.choice([True, False]))
    if op == "append":
        B = _log(rng, 1, 64)
        n_hi = _log(rng, 1, max(1, 8192 // B))
        cache = rng.choice(["bf16", "fp8"])
        return dict(op=op, cache=cache, B=B, c_lo=0, c_hi=_log(rng, 1, 4096), n_lo=1, n_hi=n_hi, Hq=G * Hkv, Hkv=Hkv,
                    d=128 if cache == "fp8" else d, rot=128 if cache == "fp8" else rng.choice([d, d // 2]),
                    axes=rng.choice([1, 2, 3]), pairs=rng.choice(["half", "adjacent"]), lens=lens)
    while True:
        n_hi = _log(rng, 1, 2048)
        B = _log(rng, 1, max(1, min(64, 8192 // n_hi)))
        c_hi = _log(rng, 16, min(131072, 1600000 // B))
        case = dict(op=op, B=B, c_lo=rng.choice([0, c_hi // 2, c_hi]), c_hi=c_hi, n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi,
                    Hq=G * Hkv, Hkv=Hkv, causal=rng.random() < 0.8, lens=lens)
        scores = B * G * Hkv * n_hi * (c_hi + n_hi)  # of the padded batch
        if scores <= 32 * 2048 * 32768 and B * (c_hi + n_hi) * Hkv <= 8 * 400000:
            return case


def _lengths(case):
    """(cached, new) token counts of the case's sequences; at least one new token in all."""
    r = random.Random(case["lens"])
    cached = [r.randint(case["c_lo"], case["c_hi"]) for _ in range(case["B"])]
    new = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    if not any(new):
        new[0] = case["n_hi"]
    return cached, new


def _blocks(n):
    return -(-n // BS)


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _ints(v, dev, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).to(dev)


def _axis_map(case):
    """Axis of each rotated pair: contiguous sections, the first axis the smallest, as image models lay them out."""
    half, A = case["rot"] // 2, case["axes"]
    if A == 1:
        return [0] * half
    first = half // (A + 1)
    rest = (half - first) // (A - 1)
    return [0] * first + [min(A - 1, 1 + (i // rest)) for i in range(half - first)]


def _axis_positions(axes, n, g, dev, base):
    """Positions [axes, n]: a running index on the first axis, and rows and columns of image patches on the others."""
    pos = [base]
    for _ in range(1, axes):
        pos.append(base // 7 + torch.randint(0, 96, (n,), generator=g, device=dev, dtype=torch.int32))
    return torch.stack(pos).to(torch.int32).contiguous()


def _codes(shape, g, dev, scale):
    """e4m3 codes (as bytes) of N(0, 1) values over the scale, made in slices so that the fp32 draw stays small."""
    out = torch.empty(shape, dtype=torch.uint8, device=dev)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 26):
        part = flat[at:at + (1 << 26)]
        x = torch.randn(part.numel(), generator=g, device=dev)
        part.copy_((x / scale).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8))
    return out


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op = case["op"]
    st = {"case": case, "op": op}
    if op in ("rope", "append"):
        half = case["rot"] // 2
        st["inv_freq"] = (ROPE_BASE ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32).to(dev)
        st["freq_axis"] = bytes(_axis_map(case))
        st["axis_index"] = _ints(_axis_map(case), dev, torch.int64)
    if op == "rope":
        n, Hq, Hkv, d = case["n"], case["Hq"], case["Hkv"], case["d"]
        start = int(torch.randint(0, 100000, (1,), generator=g, device=dev))
        st["positions"] = _axis_positions(case["axes"], n, g, dev,
                                          start + torch.arange(n, device=dev, dtype=torch.int32))
        if case["fused"]:  # q and k as columns of one projection's output, v behind them
            row = torch.randn(n, (Hq + 2 * Hkv) * d, generator=g, device=dev).to(torch.bfloat16)
            st["q"], st["k"] = row[:, :Hq * d], row[:, Hq * d:(Hq + Hkv) * d]
        else:
            st["q"] = torch.randn(n, Hq * d, generator=g, device=dev).to(torch.bfloat16)
            st["k"] = torch.randn(n, Hkv * d, generator=g, device=dev).to(torch.bfloat16)
        st["q_out"] = torch.empty(n, Hq, d, device=dev, dtype=torch.bfloat16)
        st["k_out"] = torch.empty(n, Hkv, d, device=dev, dtype=torch.bfloat16)
        return st
    cached, new = _lengths(case)
    B, total = case["B"], sum(new)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    st |= {"total": total, "cached": _ints(cached, dev), "new": _ints(new, dev)}
    if op == "plan":
        need = [_blocks(c + m) - _blocks(c) for c, m in zip(cached, new)]
        held = sum(_blocks(c) for c in cached)
        pool = held + sum(need) + 64
        ids = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        # the blocks that the cached tokens sit in, handed out in order of the sequences
        nb = _ints([_blocks(c) for c in cached], dev, torch.int64)
        off = torch.cumsum(nb, 0) - nb
        col = torch.arange(case["max_blocks"], device=dev)
        at = (off[:, None] + col[None, :]).clamp_(max=pool - 1)
        st["block_table"] = torch.where(col[None, :] < nb[:, None], ids[at], torch.full_like(ids[at], -1))
        st["free_blocks"] = ids[held:].contiguous()
        st["pos_offsets"] = torch.randint(-200, 1, (B,), generator=g, device=dev, dtype=torch.int32)
        st["max_tokens"] = total + case["pad"]
        for name, size in (("seq_lens", B), ("cu_seqlens_q", B + 1), ("slot_map", st["max_tokens"]),
                           ("positions", st["max_tokens"]), ("blocks_taken", 1)):
            st[name] = torch.empty(size, dtype=torch.int32, device=dev)
        return st
    lens = [c + m for c, m in zip(cached, new)]
    nblk = [_blocks(x) for x in lens]
    width, pool = max(nblk), sum(nblk) + 8
    ids = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    nb = _ints(nblk, dev, torch.int64)
    off = torch.cumsum(nb, 0) - nb
    col = torch.arange(width, device=dev)
    at = (off[:, None] + col[None, :]).clamp_(max=pool - 1)
    table = torch.where(col[None, :] < nb[:, None], ids[at], torch.full_like(ids[at], -1))
    cu_t = _ints(cu, dev)
    st |= {"pool": pool, "width": width, "table": table, "seq_lens": _ints(lens, dev), "cu": cu_t, "max_new": max(new),
           "max_len": max(lens)}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op == "append":
        d = case["d"]
        tok = torch.arange(total, device=dev)
        b = torch.searchsorted(cu_t[1:].long(), tok, right=True)
        pos = (st["cached"].long()[b] + tok - cu_t.long()[b])
        st["slot_map"] = (table.long()[b, pos // BS] * BS + pos % BS).to(torch.int32)
        st["positions"] = _axis_positions(case["axes"], total, g, dev, pos.to(torch.int32))
        st["qkv"] = torch.randn(total, (Hq + 2 * Hkv) * d, generator=g, device=dev).to(torch.bfloat16)
        st["q_out"] = torch.empty(total, Hq, d, device=dev, dtype=torch.bfloat16)
        if case["cache"] == "fp8":
            st["k_scale"], st["v_scale"] = 0.021, 0.017
            st["k_cache"] = _codes((pool, BS, Hkv, d), g, dev, st["k_scale"])
            st["v_cache"] = _codes((pool, BS, Hkv, d), g, dev, st["v_scale"])
        else:
            st["k_cache"] = torch.randn(pool, BS, Hkv, d, generator=g, device=dev).to(torch.bfloat16)
            st["v_cache"] = torch.randn(pool, BS, Hkv, d, generator=g, device=dev).to(torch.bfloat16)
        return st
    d = 128
    st["k_scale"], st["v_scale"], st["scale"] = 0.021, 0.017, 1.0 / math.sqrt(d)
    st["q"] = torch.randn(total, Hq, d, generator=g, device=dev).to(torch.bfloat16)
    st["k_cache"] = _codes((pool, BS, Hkv, d), g, dev, st["k_scale"])
    st["v_cache"] = _codes((pool, BS, Hkv, d), g, dev, st["v_scale"])
    st["o"] = torch.empty(total, Hq, d, device=dev, dtype=torch.bfloat16)
    st["lse"] = torch.empty(Hq, total, device=dev, dtype=torch.float32)
    return st


# ------------------------------------------------------------------ plain forms
def _plain_plan(st):
    cached, new, table = st["cached"].long(), st["new"].long(), st["block_table"]
    dev, B = table.device, cached.numel()
    seq = cached + new
    first, last = (cached + BS - 1) // BS, (seq + BS - 1) // BS
    need = last - first
    off = torch.cumsum(need, 0) - need
    free = st["free_blocks"].long()
    cu = torch.zeros(B + 1, dtype=torch.int64, device=dev)
    cu[1:] = torch.cumsum(new, 0)
    col = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (col >= first[:, None]) & (col < last[:, None])
    at = (off[:, None] + col - first[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at].to(torch.int32), table))
    tok = torch.arange(st["max_tokens"], device=dev)
    real = tok < cu[-1]
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True).clamp(max=B - 1)
    pos = torch.where(real, cached[b] + tok - cu[b], 0)
    slot = table.long()[b, (pos // BS).clamp(max=table.shape[1] - 1)] * BS + pos % BS
    i32 = torch.int32
    return {"block_table": table, "seq_lens": seq.to(i32), "cu_seqlens_q": cu.to(i32),
            "slot_map": torch.where(real, slot, -1).to(i32),
            "positions": torch.where(real, pos + st["pos_offsets"].long()[b], 0).to(i32),
            "blocks_taken": need.sum().reshape(1).to(i32)}


def _plain_angles(st):
    # far positions lose their angle in 32 bits
    a = st["positions"][st["axis_index"]].t().double() * st["inv_freq"].double()
    return a.cos().float(), a.sin().float()


def _plain_rotate(x, H, d, rot, pairs, cos, sin):
    """x [n, H * d] (any row stride) -> fp32 [n, H, d] with the first `rot` of each head rotated."""
    x = x.reshape(x.shape[0], H, d).float()
    r, rest = x[..., :rot], x[..., rot:]
    c, s = cos[:, None, :], sin[:, None, :]
    if pairs == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _plain_rope(st):
    c = st["case"]
    cos, sin = _plain_angles(st)
    if c["dir"] == "bwd":
        sin = -sin
    return {"q": _plain_rotate(st["q"], c["Hq"], c["d"], c["rot"], c["pairs"], cos, sin).to(torch.bfloat16),
            "k": _plain_rotate(st["k"], c["Hkv"], c["d"], c["rot"], c["pairs"], cos, sin).to(torch.bfloat16)}


def _split_qkv(st):
    c = st["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    row = st["qkv"]
    return row[:, :Hq * d], row[:, Hq * d:(Hq + Hkv) * d], row[:, (Hq + Hkv) * d:]


def _plain_append(st):
    c = st["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    q, k, v = _split_qkv(st)
    cos, sin = _plain_angles(st)
    q_out = _plain_rotate(q, Hq, d, c["rot"], c["pairs"], cos, sin).to(torch.bfloat16)
    k = _plain_rotate(k, Hkv, d, c["rot"], c["pairs"], cos, sin)
    v = v.reshape(-1, Hkv, d).float()
    slots = st["slot_map"].long()
    if c["cache"] == "fp8":
        k = (k / st["k_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
        v = (v / st["v_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    st["k_cache"].view(-1, Hkv, d)[slots] = k
    st["v_cache"].view(-1, Hkv, d)[slots] = v
    return {"q": q_out, **_caches(st)}


def _caches(st):
    """The caches as the values they hold (FP8 codes as FP8 numbers)."""
    k, v = st["k_cache"], st["v_cache"]
    return {"k_cache": k.view(E4M3) if k.dtype == torch.uint8 else k,
            "v_cache": v.view(E4M3) if v.dtype == torch.uint8 else v}


def _plain_chunk(st):
    c = st["case"]
    B, Hq, Hkv, T, S, d = c["B"], c["Hq"], c["Hkv"], st["max_new"], st["max_len"], 128
    G, dev = Hq // Hkv, st["q"].device
    cu, lens = st["cu"].long(), st["seq_lens"].long()
    n_new = cu[1:] - cu[:-1]
    # queries padded to [B, Hkv, G * T, d], keys and values gathered through the table to [B, Hkv, S, d]
    i = torch.arange(T, device=dev)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=st["total"] - 1)
    q = st["q"].float()[rows].view(B, T, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, d)
    blocks = st["table"].long().clamp(min=0)
    k = st["k_cache"].view(E4M3)[blocks].float().view(B, -1, Hkv, d)[:, :S].permute(0, 2, 3, 1)
    v = st["v_cache"].view(E4M3)[blocks].float().view(B, -1, Hkv, d)[:, :S].permute(0, 2, 1, 3)
    s = torch.matmul(q, k * st["k_scale"]).view(B, Hkv, G, T, S) * st["scale"]
    j = torch.arange(S, device=dev)
    limit = lens[:, None] - n_new[:, None] + i[None, :] if c["causal"] else (lens[:, None] - 1).expand(B, T)
    seen = (j[None, None, :] <= limit[:, :, None]) & (j[None, None, :] < lens[:, None, None])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * T, S), v * st["v_scale"]).view(B, Hkv, G, T, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).view(B, Hq, T)
    tok = torch.arange(st["total"], device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    at = tok - cu[b]
    o = o.view(B, Hq, T, d).permute(0, 2, 1, 3)[b, at]
    return {"o": o.to(torch.bfloat16), "lse": lse.permute(0, 2, 1)[b, at].t().contiguous()}


# ------------------------------------------------------------------ the library's calls
def _own(st):
    import flashattention_attention_attn_b200 as fa

    c, op = st["case"], st["op"]
    if op == "plan":
        fa.paged_cache_plan(st["cached"], st["new"], st["free_blocks"], st["pos_offsets"], c["B"],
                            st["free_blocks"].numel(), BS, c["max_blocks"], st["max_tokens"], st["block_table"],
                            st["seq_lens"], st["cu_seqlens_q"], st["slot_map"], st["positions"], st["blocks_taken"])
        return {k: st[k] for k in ("block_table", "seq_lens", "cu_seqlens_q", "slot_map", "positions", "blocks_taken")}
    if op == "rope":
        call = fa.rope_axes_fwd if c["dir"] == "fwd" else fa.rope_axes_bwd
        Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
        call(st["q"], st["k"], st["positions"], st["inv_freq"], st["freq_axis"], c["n"], Hq, Hkv, d, c["rot"], c["axes"],
             st["positions"].stride(0), st["q"].stride(0), st["k"].stride(0), c["pairs"] == "adjacent", st["q_out"],
             st["k_out"], Hq * d, Hkv * d)
        return {"q": st["q_out"], "k": st["k_out"]}
    if op == "append":
        q, k, v = _split_qkv(st)
        args = (q, k, v, st["positions"], st["inv_freq"], st["freq_axis"], st["slot_map"], st["total"], c["Hq"], c["Hkv"],
                c["d"], c["rot"], c["axes"], st["positions"].stride(0), q.stride(0), k.stride(0), v.stride(0),
                c["pairs"] == "adjacent", BS, st["pool"])
        if c["cache"] == "fp8":
            fa.rope_axes_paged_append_fp8(*args, st["k_scale"], st["v_scale"], st["q_out"], st["k_cache"], st["v_cache"])
        else:
            fa.rope_axes_paged_append(*args, st["q_out"], st["k_cache"], st["v_cache"])
        return {"q": st["q_out"], **_caches(st)}
    fa.paged_attn_prefill_fp8_checked(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq_lens"], st["cu"], c["B"],
                                      c["Hq"], c["Hkv"], 128, BS, st["width"], st["pool"], st["max_new"], st["total"],
                                      c["causal"], st["scale"], st["k_scale"], st["v_scale"], 0, st["o"], st["lse"])
    return {"o": st["o"], "lse": st["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "rope": _plain_rope, "append": _plain_append, "chunk": _plain_chunk}[state["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rotate(x, angle, rot, adjacent, sign):
    """Complex numbers: each pair times exp(sign * i * angle); x [n, H, d] and angle [n, rot / 2] in 64 bits."""
    y = x.clone()
    even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., even], x[..., odd]) * torch.polar(torch.ones_like(angle), sign * angle)[:, None, :]
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    st = prepare(case, seed)
    f64 = torch.float64
    if op in ("rope", "append"):
        pos = torch.stack([st["positions"][a] for a in st["freq_axis"]], 1).to(f64)
        angle = pos * st["inv_freq"].to(f64)[None, :]
        adjacent, Hq, Hkv, d, rot = case["pairs"] == "adjacent", case["Hq"], case["Hkv"], case["d"], case["rot"]
    if op == "rope":
        sign = 1.0 if case["dir"] == "fwd" else -1.0
        return {"q": _exact_rotate(st["q"].to(f64).view(-1, Hq, d), angle, rot, adjacent, sign),
                "k": _exact_rotate(st["k"].to(f64).view(-1, Hkv, d), angle, rot, adjacent, sign)}
    if op == "append":
        q, k, v = (x.to(f64) for x in _split_qkv(st))
        k = _exact_rotate(k.view(-1, Hkv, d), angle, rot, adjacent, 1.0)
        v = v.view(-1, Hkv, d)
        kc, vc = _caches(st)["k_cache"].to(f64), _caches(st)["v_cache"].to(f64)
        if case["cache"] == "fp8":
            k, v = k / st["k_scale"], v / st["v_scale"]
        kc.view(-1, Hkv, d).index_copy_(0, st["slot_map"].long(), k)
        vc.view(-1, Hkv, d).index_copy_(0, st["slot_map"].long(), v)
        return {"q": _exact_rotate(q.view(-1, Hq, d), angle, rot, adjacent, 1.0), "k_cache": kc, "v_cache": vc}
    cached, new = _lengths(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    if sum(4.0 * 128 * Hq * m * (c + m) for c, m in zip(cached, new)) > 4e13:
        return None
    o = torch.zeros(st["total"], Hq, 128, dtype=f64, device=st["q"].device)
    lse = torch.full((Hq, st["total"]), -math.inf, dtype=f64, device=st["q"].device)
    at = 0
    for b, (c, m) in enumerate(zip(cached, new)):
        if m == 0:
            continue
        ids = st["table"][b, :_blocks(c + m)].long()
        for h in range(Hkv):
            K = st["k_cache"][ids][:, :, h].view(E4M3).to(f64).reshape(-1, 128)[:c + m] * st["k_scale"]
            V = st["v_cache"][ids][:, :, h].view(E4M3).to(f64).reshape(-1, 128)[:c + m] * st["v_scale"]
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                s = (st["q"][at:at + m, g].to(f64) @ K.T) * st["scale"]
                if case["causal"]:
                    s += torch.full_like(s, -math.inf).triu(c + 1)
                lse[g, at:at + m] = torch.logsumexp(s, 1)
                o[at:at + m, g] = torch.softmax(s, 1) @ V
        at += m
    return {"o": o, "lse": lse}


def work(case):
    """Each input read once, each output written once; two operations for every product and sum."""
    op = case["op"]
    if op == "rope":
        n, H, d = case["n"], case["Hq"] + case["Hkv"], case["d"]
        return {"bytes": 2 * 2 * n * H * d + 4 * n * case["axes"] + 2 * case["rot"], "flops": 3 * n * H * case["rot"]}
    cached, new = _lengths(case)
    total = sum(new)
    if op == "plan":
        need = sum(_blocks(c + m) - _blocks(c) for c, m in zip(cached, new))
        part = sum(1 for c, m in zip(cached, new) if m and c % BS)
        return {"bytes": 4 * (3 * case["B"] + part + need) + 4 * (need + 2 * case["B"] + 2 + 2 * (total + case["pad"])),
                "flops": 0}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op == "append":
        d, size = case["d"], 1 if case["cache"] == "fp8" else 2
        rows = total * d
        return {"bytes": rows * (2 * (Hq + 2 * Hkv) + 2 * Hq + 2 * Hkv * size) + 4 * total * (case["axes"] + 1) +
                2 * case["rot"], "flops": 3 * total * (Hq + Hkv) * case["rot"]}
    pairs = sum(m * c + m * (m + 1) // 2 if case["causal"] else m * (c + m) for c, m in zip(cached, new))
    keys = sum(c + m for c, m in zip(cached, new) if m)
    return {"bytes": 2 * keys * Hkv * 128 + 2 * 2 * total * Hq * 128 + 4 * Hq * total +
            4 * sum(_blocks(c + m) for c, m in zip(cached, new) if m) + 8 * case["B"], "flops": 4 * 128 * Hq * pairs}
