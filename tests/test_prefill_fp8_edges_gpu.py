"""paged_attn_prefill_fp8 at the edges of what its documentation allows."""

import pytest
import torch

from flashattention_attention_attn_b200 import inputs
from tests.test_prefill_fp8_gpu import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx,ql", [([10, 200], [40, 3]), ([3, 50], [8, 2]), ([2, 20], [4, 1])])
@pytest.mark.parametrize("splits", [0, 1, 2])
def test_a_row_that_sees_no_key_is_empty_whatever_its_query_holds(ctx, ql, splits):
    """Causal, more queries than keys: the first rows see nothing, o = 0 and lse = -inf, also where q is NaN or infinite
    (the sums run over no key); the rows that see keys are as before, and NaN where their own q is."""
    q, cu, c, scale = make(ctx, ql, Hq=8, Hkv=2, seed=13)
    want = run(q, cu, c, True, scale, splits=splits)
    q2 = q.clone()
    q2[0, 3, 7], q2[0, 1, 0], q2[0, 2, 5] = float("nan"), float("inf"), float("-inf")
    q2[ql[0] - 1, 0, 0], q2[ql[0] - 1, 5, 9] = float("nan"), float("inf")  # the last row sees every key
    o, lse, st = run(q2, cu, c, True, scale, splits=splits)
    assert st == 0
    assert torch.all(o[0] == 0) and torch.all(lse[:, 0] == float("-inf"))
    hit = torch.zeros(q.shape[:2], dtype=torch.bool)
    hit[ql[0] - 1, 0] = hit[ql[0] - 1, 5] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse.t()[hit]).all()
    assert torch.equal(o[~hit], want[0][~hit]) and torch.equal(lse.t()[~hit], want[1].t()[~hit])


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
