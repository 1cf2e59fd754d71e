"""Plain CPU oracle of the serving step around the paged cache: the plan of a
step, rotary positions with several axes, and the cache write.

TEST INFRASTRUCTURE ONLY, like fp64_attention: nothing here is shared with the
library, and this module imports nothing from it.  Whole numbers are Python
loops over the definition; rotations are fp64 numpy.

The block table is the one of the page "Snelle attention-kernels en
operatorfusie versnellen AI-modellen" (the-ai.news), section
"FlashAttention-type aandacht en gepagineerde aandacht": fixed-size blocks and
a table that maps every logical position to a physical block.
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["plan_step", "rope_axes", "append_slots", "e4m3_values", "nearest_e4m3"]

BLOCK = 16
MAX_BLOCKS = (1 << 27) - 1  # ids from here on are no blocks


def plan_step(cached, new, free, offsets, table, max_tokens):
    """Returns a dict of the plan's outputs plus "flags", a set of "seqlen",
    "noblock" and "badblock".  `table` [B, max_blocks] is not modified."""
    table = np.array(table, dtype=np.int64)
    B = len(cached)
    cap = (table.shape[1] if B else 0) * BLOCK
    flags, lens, cu, slots, positions = set(), [], [0], [], []
    taken = 0
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        if c < 0 or n < 0 or c + n > cap:
            flags.add("seqlen")
        c, n = min(max(c, 0), cap), max(n, 0)
        if n > max_tokens - cu[-1]:
            flags.add("seqlen")
            n = max_tokens - cu[-1]
        length = min(c + n, cap)
        lens.append(length)
        cu.append(cu[-1] + n)
        short = set()  # blocks that found no free id
        for j in range(-(-c // BLOCK), -(-length // BLOCK)):
            if taken < len(free):
                table[b, j] = int(free[taken])
            else:
                table[b, j] = -1
                short.add(j)
                flags.add("noblock")
            taken += 1
        for p in range(c, c + n):
            slot = -1
            if p < cap:
                block = int(table[b, p // BLOCK])
                if 0 <= block < MAX_BLOCKS:
                    slot = block * BLOCK + p % BLOCK
                elif p // BLOCK not in short:
                    flags.add("badblock")
            slots.append(slot)
            positions.append(p + (int(offsets[b]) if offsets is not None else 0))
    pad = max_tokens - len(slots)
    return {"block_table": table.astype(np.int32), "seq_lens": np.array(lens, dtype=np.int32),
            "cu_seqlens_q": np.array(cu, dtype=np.int32), "slot_map": np.array(slots + [-1] * pad, dtype=np.int32),
            "positions": np.array(positions + [0] * pad, dtype=np.int32),
            "blocks_taken": np.array([taken], dtype=np.int32), "flags": flags}


def rope_axes(x, positions, inv_freq, freq_axis, adjacent, sign=1.0):
    """x [n, H, d] fp64, positions [axes, n], inv_freq [half] (the fp32 numbers
    as fp64), freq_axis [half]: the first 2 * half elements of every head
    rotated by sign * positions[freq_axis[i], t] * inv_freq[i]."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    y = x.copy()
    for i in range(half):
        phi = sign * np.asarray(positions[freq_axis[i]], dtype=np.float64) * float(inv_freq[i])
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
        e, o = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        y[..., e] = x[..., e] * c - x[..., o] * s
        y[..., o] = x[..., o] * c + x[..., e] * s
    return y


def append_slots(cache, rows, slots):
    """cache [pool, 16, Hkv, d] with rows[t] at slot slots[t]; negative slots
    and slots past the pool are dropped."""
    out = np.array(cache)
    for t, s in enumerate(slots):
        if 0 <= s < out.shape[0] * BLOCK:
            out[s // BLOCK, s % BLOCK] = rows[t]
    return out


def e4m3_values():
    """The 127 non-negative finite e4m3 values, ascending (code = index)."""
    v = [math.ldexp(m / 8.0, -6) for m in range(8)]
    v += [math.ldexp(1.0 + m / 8.0, e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:127])


def nearest_e4m3(x):
    """Codes of the nearest e4m3 values (ties to the even code, saturated),
    by search in the table of values."""
    v = e4m3_values()
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), v[-1])
    hi = np.clip(np.searchsorted(v, a), 1, 126)
    lo = hi - 1
    up = (a - v[lo] > v[hi] - a) | ((a - v[lo] == v[hi] - a) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)
