"""paged_cache_plan against the oracle's loops: every output equal, nothing
else written."""

import numpy as np
import pytest
import torch

from oracle import paged_step as ps

pytestmark = pytest.mark.gpu
FLAGS = {"badblock": 0x2, "seqlen": 0x4, "noblock": 0x8}


def plan(cached, new, free, offsets, table, max_tokens, stream=None):
    """Runs the call on guarded buffers; returns the outputs and the status word."""
    import flashattention_attention_attn_b200 as fa
    B = len(cached)
    i32 = dict(dtype=torch.int32, device="cuda")
    max_blocks = table.shape[1] if B else 1
    tab = torch.tensor(np.asarray(table), **i32) if B else None
    out = {"seq_lens": B, "cu_seqlens_q": B + 1, "slot_map": max_tokens, "positions": max_tokens, "blocks_taken": 1}
    buf = {k: torch.full((n + 8,), -77, **i32) for k, n in out.items()}
    t = [torch.tensor(x, **i32) if x is not None else None for x in (cached, new, free, offsets)]
    fa.paged_cache_plan(*t, B, len(free), 16, max_blocks, max_tokens, tab, buf["seq_lens"], buf["cu_seqlens_q"],
                        buf["slot_map"], buf["positions"], buf["blocks_taken"], stream)
    torch.cuda.synchronize()
    got = {k: buf[k][:n].cpu().numpy() for k, n in out.items()}
    for k, n in out.items():
        assert torch.all(buf[k][n:] == -77), k
    got["block_table"] = tab.cpu().numpy() if B else np.zeros((0, 0), dtype=np.int32)
    return got, fa.attn_read_device_status(clear=True)


def check(cached, new, free, offsets, table, max_tokens):
    want = ps.plan_step(cached, new, free, offsets, table, max_tokens)
    got, status = plan(cached, new, free, offsets, table, max_tokens)
    for k in got:
        if k != "block_table" or len(cached):
            assert np.array_equal(got[k], want[k]), k
    assert status == sum(FLAGS[f] for f in want["flags"])
    return got


def batch(seed, B, c_hi, n_hi, max_blocks=None):
    g = np.random.default_rng(seed)
    cached, new = g.integers(0, c_hi + 1, B), g.integers(0, n_hi + 1, B)
    width = max_blocks or (c_hi + n_hi) // 16 + 1
    held = -(-cached // 16)
    ids = g.permutation(int(held.sum()) + B * (n_hi // 16 + 2))
    table = np.full((B, width), -1)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    return cached.tolist(), new.tolist(), ids[at:].tolist(), g.integers(-50, 50, B).tolist(), table


@pytest.mark.parametrize("B,c_hi,n_hi", [(1, 0, 1), (1, 100, 1), (3, 40, 17), (64, 500, 1), (33, 0, 2000), (511, 64, 40),
                                         (512, 64, 3), (513, 64, 40), (2000, 33, 9)])
@pytest.mark.parametrize("pad", [0, 77])
def test_batches(B, c_hi, n_hi, pad):
    cached, new, free, offsets, table = batch(B + n_hi, B, c_hi, n_hi)
    check(cached, new, free, offsets if pad else None, table, sum(new) + pad)


def test_one_long_prompt_takes_many_blocks():
    cached, new, free, _, table = [0, 131], [50001, 0], list(range(5000)), None, np.full((2, 4000), -1)
    table[1, :9] = range(6000, 6009)
    check(cached, new, free, None, table, 50001 + 7)


def test_empty_sequences_at_both_ends_and_in_runs():
    cached, new, free, offsets, table = batch(5, 40, 60, 30)
    new = [n if 5 < i < 9 or i == 30 else 0 for i, n in enumerate(new)]
    check(cached, new, free, offsets, table, sum(new))
    check(cached, [0] * 40, free, offsets, table, 5)


def test_no_sequences():
    got = check([], [], [3, 4], None, np.zeros((0, 1)), 9)
    assert got["slot_map"].tolist() == [-1] * 9 and got["cu_seqlens_q"].tolist() == [0]
    check([], [], [], None, np.zeros((0, 1)), 0)


def test_malformed_lengths_and_short_lists():
    cached, new, free, offsets, table = batch(9, 50, 60, 40, max_blocks=9)
    check(cached, new, free[:11], offsets, table, sum(new))               # the free list runs out
    check(cached, new, free, offsets, table, sum(new) // 3)               # more rows than the buffers take
    bad = [c if i % 7 else -3 for i, c in enumerate(cached)]
    check(bad, [n if i % 5 else -n - 1 for i, n in enumerate(new)], free, offsets, table, 4000)
    check([c + 100 * (i == 20) for i, c in enumerate(cached)], new, free, offsets, table, 4000)  # past the table row
    check([3, 20], [2, 2], [], None, np.array([[-1, -1], [8, 1 << 27]]), 6)  # last blocks that are no blocks
    check([0], [20], [-5, 2], None, np.array([[-1, -1]]), 20)
    check([2**31 - 1, 5], [2**31 - 1, 3], [1], None, np.array([[4, 5], [6, 7]]), 12)


def test_a_second_step_continues_the_first():
    """Two steps as a server makes them: the table, with the taken ids dropped, serves the next step."""
    cached, new, free, _, table = batch(11, 37, 90, 50, max_blocks=30)
    a = check(cached, new, free, None, table, sum(new))
    n = int(a["blocks_taken"][0])
    b = check(a["seq_lens"].tolist(), [1] * 37, free[n:], None, a["block_table"], 37)
    assert len(set(b["slot_map"].tolist() + a["slot_map"].tolist())) == sum(new) + 37


def test_captured_and_replayed_with_new_lengths():
    import flashattention_attention_attn_b200 as fa
    i32 = dict(dtype=torch.int32, device="cuda")
    B, width, cap = 20, 12, 512
    cached, new = torch.zeros(B, **i32), torch.ones(B, **i32)
    free, table = torch.arange(400, **i32), torch.full((B, width), -1, **i32)
    lens, cu, slots, pos, taken = (torch.empty(n, **i32) for n in (B, B + 1, cap, cap, 1))

    def call():
        fa.paged_cache_plan(cached, new, free, None, B, 400, 16, width, cap, table, lens, cu, slots, pos, taken)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in range(3):
        c, n, f, _, t = batch(seed, B, 60, 20, max_blocks=width)
        f = (f + [999] * 400)[:400]
        for dst, src in ((cached, c), (new, n), (free, f), (table, t)):
            dst.copy_(torch.tensor(np.asarray(src), **i32))
        want = ps.plan_step(c, n, f, None, t, cap)
        g.replay()
        torch.cuda.synchronize()
        for k, v in (("block_table", table), ("seq_lens", lens), ("cu_seqlens_q", cu), ("slot_map", slots),
                     ("positions", pos), ("blocks_taken", taken)):
            assert np.array_equal(v.cpu().numpy(), want[k]), k
    assert fa.attn_read_device_status(clear=True) == 0
