"""paged_attn_prefill_fp8 at the edges of what its documentation allows."""

import pytest
import torch

from flashattention_attention_attn_b200 import inputs
from tests.test_prefill_fp8_gpu import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("splits", [0, 1, 2])
def test_a_table_wider_than_2_to_26_blocks(T, splits):
    """max_blocks up to 2^27 is supported, for few rows and for many: only the entries that the length needs are read
    (with two ranges all keys lie on the first)."""
    q, cu, c, scale = make([300], [T], Hq=8, Hkv=2, seed=17)
    wide = torch.full((1, (1 << 26) + 40), -1, dtype=torch.int32)
    wide[:, :c.block_table.shape[1]] = c.block_table
    e = inputs.PagedInputsFp8(c.q, c.k_cache, c.v_cache, wide, c.seq_lens, 16, c.k_scale, c.v_scale)
    o, lse, st = run(q, cu, e, True, scale, splits=splits)
    assert st == 0
    check(q, cu, c, True, scale, o, lse)
