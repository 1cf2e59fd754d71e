"""The serving step's limits and refusals at their borders, without a GPU."""

import pytest
import torch

from tests.test_paged_step_host import INVALID, UNSUPPORTED, _append, _chunk, _without_device, lib  # noqa: F401 (lib is a fixture)

WIDE = (1 << 27) - 1  # the widest table: 2^24 tiles of 128 keys


@pytest.mark.parametrize("kw,refused", [
    (dict(B=127, maxb=WIDE, max_q=4), False),                 # few rows: 127 (2^24 + 3) < 2^31 - 2^20
    (dict(B=128, maxb=WIDE, max_q=4), True),
    (dict(B=128, maxb=WIDE, max_q=8, splits=1), True),
    (dict(B=127, maxb=WIDE, max_q=8, splits=1 << 23), False),
    (dict(B=100, maxb=(1 << 27) - 8, max_q=8, splits=(1 << 23) + 5), False),  # ranges of two tiles: as long as the row
    (dict(B=128, maxb=WIDE - 8, max_q=8, splits=(1 << 24) - 2), True),
    (dict(B=128, maxb=WIDE, max_q=9), False),                 # many rows
    (dict(B=1, maxb=WIDE, max_q=40), False),
    (dict(B=128, maxb=WIDE, max_q=40, total_q=8), True),      # no more rows than total_q: few
])
def test_chunk_attention_takes_wide_tables_up_to_the_stated_limit(lib, kw, refused):  # noqa: F811
    if not refused and torch.cuda.is_available():
        pytest.skip("the addresses of an accepted call are made up")
    rc = _chunk(lib, **kw)
    assert rc == UNSUPPORTED if refused else _without_device(rc)


@pytest.mark.parametrize("scales,refused", [
    ((2.0 ** -130, 1.0), True),      # the reciprocal is infinite in fp32: zeros would become NaN codes
    ((1.0, 2.0 ** -149), True),
    ((2.0 ** -128, 1.0), True),
    ((2.0 ** -127, 2.0 ** -126), False),
    ((3e38, 1.0), False),
])
def test_append_fp8_refuses_scales_without_a_reciprocal(lib, scales, refused):  # noqa: F811
    if not refused and torch.cuda.is_available():
        pytest.skip("the addresses of an accepted call are made up")
    rc = _append(lib, fp8=True, scales=scales)
    assert rc == INVALID if refused else _without_device(rc)


def test_rope_op_refuses_frequencies_that_want_a_gradient():
    """None is computed for them, so a call that would leave it out silently is refused; q and k alone train."""
    import flashattention_attention_attn_b200.torch_ops  # noqa: F401
    rope = torch.ops.fa_b200.rope_axes
    with torch._subclasses.FakeTensorMode():
        q, k = (torch.empty(5, h, 64, dtype=torch.bfloat16, requires_grad=True) for h in (4, 2))
        f, pos = torch.empty(32, requires_grad=True), torch.empty(1, 5, dtype=torch.int32)
        with pytest.raises(ValueError, match="inv_freq"):
            rope(q, k, pos, f, [], False)
        with pytest.raises(ValueError, match="inv_freq"):
            rope(q.detach(), k.detach(), pos, f, [], False)
        a, b = rope(q, k, pos, f.detach(), [], False)
        dq, dk = torch.autograd.grad((a, b), (q, k), (torch.empty_like(a), torch.empty_like(b)))
        assert dq.shape == q.shape and dk.shape == k.shape
        with torch.no_grad():
            assert rope(q, k, pos, f, [], False)[0].shape == q.shape
