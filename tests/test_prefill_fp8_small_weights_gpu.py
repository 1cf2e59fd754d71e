"""paged_attn_prefill_fp8 where the small weights of a long row decide its result: a key far above all others (an
attention sink) whose value is zero, before up to 131072 keys whose weights are 2^-17 to 2^-22 of its.

Every row of q is the same and sees every key, so the definition is one softmax over the sequence in 64 bits.

Tolerance.  The score products are exact (ones times few-bit numbers).  A weight is off by half an f16 step, 2^-11 of
itself or 2^-25 where the f16 is subnormal; the row's largest is at least 2^6, so the latter is 2^-31 of the sum of the
weights at most, for each of N keys.  The exponent's fp32 roundings (a scale of two products, a multiply-add near 2^5)
move a weight by 2^-16 at most, the row sum's N / 128 additions the sum by N / 128 * 2^-24, the tensor core's N / 16
additions the product by N / 16 * 2^-23 (it may truncate); o is rounded to bf16, 2^-8 of the value.  With values of 0
and 1:  |d o| <= (2^-8 + 2^-11 + 2^-16 + N 2^-31 + N 2^-27) |o| + N 2^-31."""

import numpy as np
import pytest
import torch

from flashattention_attention_attn_b200 import inputs
from oracle import fp64_attention as orc
from tests.test_prefill_fp8_gpu import run

pytestmark = pytest.mark.gpu


def sink_case(S, gap, T, spread, Hq=4):
    """One sequence of S keys: key 0 scores `gap` (log2) above the others' lowest."""
    width = S // 16
    spec = inputs.DecodeSpec(B=1, Hq=1, Hkv=1, d=128, block_size=16, max_blocks=width, ctx_lo=1, ctx_hi=1, seed=3)
    c = inputs.make_paged_fp8(spec, seq_lens=[S], k_scale=1.0, v_scale=1.0)
    first = int(c.block_table[0, 0])
    c.k_cache[:] = 0
    if spread:  # eight elements of 0 to 7 / 8: the others' scores lie within a nat or so
        g = torch.Generator().manual_seed(7)
        codes = torch.tensor([0x00, 0x20, 0x28, 0x2C, 0x30, 0x32, 0x34, 0x36], dtype=torch.uint8)
        c.k_cache[..., 120:] = codes[torch.randint(0, 8, (*c.k_cache.shape[:3], 8), generator=g)]
    c.k_cache[first, 0, 0] = 0
    c.k_cache[first, 0, 0, :72] = 0x38  # 72 ones
    c.v_cache[:] = 0x38  # ones: o is the small weights' share
    c.v_cache[first, 0] = 0
    q = torch.ones(T, Hq, 128, dtype=torch.bfloat16)
    return q, torch.tensor([0, T], dtype=torch.int32), c, float(np.float32(gap * np.log(2.0) / 72))


def check_sink(q, cu, c, scale, o, lse):
    S = int(c.seq_lens[0])
    K = orc.decode_e4m3(c.k_cache.numpy())[c.block_table[0].numpy()].reshape(-1, 128)[:S]
    V = orc.decode_e4m3(c.v_cache.numpy())[c.block_table[0].numpy()].reshape(-1, 128)[:S]
    s = K.sum(1) * scale
    w = np.exp(s - s.max())
    want, want_lse = (w @ V) / w.sum(), s.max() + np.log(w.sum())
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16 + S * 2.0 ** -31 + S * 2.0 ** -27) * want + S * 2.0 ** -31
    err = np.abs(o.double().numpy() - want)
    assert np.all(err <= tol), (float((err / tol).max()), float(o.double().min()), float(want[0]))
    assert np.all(np.abs(lse.double().numpy() - want_lse) <= 2.0 ** -16 * 2 + S * 2.0 ** -31 + 2.0 ** -20 * abs(want_lse))


@pytest.mark.parametrize("S,gap", [(32768, 17.3), (131072, 17.3), (32768, 20.2), (131072, 20.2), (131072, 21.6)])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("T", [2, 8])
def test_few_rows_keep_small_weights(S, gap, spread, T):
    a = sink_case(S, gap, T, spread)
    for splits in (1, 0):
        o, lse, st = run(*a[:3], False, a[3], splits=splits)
        assert st == 0
        check_sink(*a, o, lse)


@pytest.mark.parametrize("S,gap", [(131072, 17.3), (32768, 20.2), (131072, 20.2), (131072, 21.6)])
@pytest.mark.parametrize("spread", [False, True])
def test_many_rows_keep_small_weights(S, gap, spread):
    a = sink_case(S, gap, 40, spread)
    for splits in (1, 0):
        o, lse, st = run(*a[:3], False, a[3], splits=splits)
        assert st == 0
        check_sink(*a, o, lse)
