"""paged_attn_prefill_fp8 against the fp64 oracle on the decoded cache.

Tolerances.  A score's error: q enters as two e4m3 terms, off by at most 2^-18
of the row's largest element, times the keys' absolute sum; 128 products are
summed in fp32 by the tensor cores, bounded by 128 * 2^-23 of the absolute
products' sum.  With d the larger of the two sums over the visible keys, times
scale: |d lse| <= d + 2^-20 |lse| + 2^-20 (ex2, log2 and the fp32 sums), and
weights move by 2 d at most and are rounded to f16 (2^-11) and o to bf16 (2^-8
of the value): |d o| <= 2^-8 |o| + (2^-11 + 2 d + 2^-18) max |v|."""

import numpy as np
import pytest
import torch

from flashattention_attention_attn_b200 import inputs
from oracle import fp64_attention as orc
from tests._parity import f64

pytestmark = pytest.mark.gpu


def make(ctx, ql, Hq=32, Hkv=8, seed=0, k_scale=0.021, v_scale=0.37, max_blocks=None, spare=3):
    width = max_blocks or max(1, max(-(-c // 16) for c in ctx))
    spec = inputs.ChunkedSpec(B=len(ctx), Hq=Hq, Hkv=Hkv, d=128, block_size=16, max_blocks=width, ctx_lo=1, ctx_hi=1,
                              q_lo=1, q_hi=1, seed=seed)
    dspec = inputs.DecodeSpec(B=len(ctx), Hq=1, Hkv=Hkv, d=128, block_size=16, max_blocks=width, ctx_lo=1, ctx_hi=1,
                              seed=seed, extra_pool_blocks=spare)
    c = inputs.make_paged_fp8(dspec, seq_lens=ctx, k_scale=k_scale, v_scale=v_scale)
    # codes over the whole range: N(0, 1) values over the scale
    g = torch.Generator().manual_seed(seed + 1)
    for name, s in (("k_cache", k_scale), ("v_cache", v_scale)):
        x = torch.randn(c.k_cache.shape, generator=g) / s
        setattr(c, name, x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    cu = torch.tensor([0] + list(np.cumsum(ql)), dtype=torch.int32)
    q = torch.randn(int(cu[-1]), Hq, 128, generator=g).to(torch.bfloat16)
    return q, cu, c, spec.scale


def run(q, cu, c, causal, scale, splits=0, num_blocks=None, lse=True, max_q=None, pad=0, stream=None):
    import flashattention_attention_attn_b200 as fa
    total, Hq, d = q.shape
    B, width = c.block_table.shape
    Hkv = c.k_cache.shape[2]
    dq = torch.cat([q, torch.randn(pad, Hq, d).to(q.dtype)]).cuda() if pad else q.cuda()
    o = torch.full_like(dq, float("nan"))
    L = torch.full((Hq, total + pad), float("nan"), device="cuda") if lse else None
    mq = int((cu[1:] - cu[:-1]).max()) if max_q is None else max_q
    head = (dq, c.k_cache.cuda(), c.v_cache.cuda(), c.block_table.cuda(), c.seq_lens.cuda(), cu.cuda(), B, Hq, Hkv, d, 16,
            width)
    tail = (mq, total + pad, causal, scale, c.k_scale, c.v_scale, splits, o, L)
    if num_blocks is None:
        fa.paged_attn_prefill_fp8(*head, *tail)
    else:
        fa.paged_attn_prefill_fp8_checked(*head, num_blocks, *tail)
    torch.cuda.synchronize()
    if pad:  # rows behind the last sequence as they were
        assert torch.isnan(o[total:]).all() and (L is None or torch.isnan(L[:, total:]).all())
    return o[:total].cpu(), (L[:, :total].cpu() if lse else None), fa.attn_read_device_status(clear=True)


def check(q, cu, c, causal, scale, o, lse, num_blocks=None):
    K = np.float32(c.k_scale).astype(np.float64) * orc.decode_e4m3(c.k_cache.numpy())
    V = np.float32(c.v_scale).astype(np.float64) * orc.decode_e4m3(c.v_cache.numpy())
    Q = f64(q)
    O, L = orc.paged_prefill(Q, K, V, c.block_table.numpy(), c.seq_lens.numpy(), cu.numpy(), 16, scale, causal,
                             num_blocks=num_blocks)
    G = q.shape[1] // c.k_cache.shape[2]
    got_o, got_l = f64(o), None if lse is None else f64(lse)
    for b in range(len(cu) - 1):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        if r0 == r1:
            continue
        Kb, Vb = orc.gather_paged_kv(K, V, c.block_table.numpy()[b], c.seq_lens.numpy()[b], 16, num_blocks)
        if Kb.shape[0] == 0:
            assert np.all(got_o[r0:r1] == 0) and (got_l is None or np.all(np.isneginf(got_l[:, r0:r1])))
            continue
        Ka = np.repeat(np.abs(Kb), G, axis=1)                        # [S, Hq, d]
        Qa = np.abs(Q[r0:r1])                                        # [T, Hq, d]
        split = 2.0 ** -18 * Qa.max(-1) * Ka.sum(-1).max(0)[None]     # [T, Hq]
        dots = np.einsum("thd,hd->th", Qa, Ka.max(0))                # over every key, an upper bound
        d = scale * (split + 128 * 2.0 ** -23 * dots)
        vmax = np.repeat(np.abs(Vb).max((0, 2)), G)[None]
        tol = 2.0 ** -8 * np.abs(O[r0:r1]) + ((2.0 ** -11 + 2 * d + 2.0 ** -18) * vmax)[..., None]
        err = np.abs(got_o[r0:r1] - O[r0:r1])
        assert np.all(err <= tol), (b, float((err / tol).max()))
        if got_l is not None:
            Lb = L[:, r0:r1]
            fin = np.isfinite(Lb)
            assert np.array_equal(np.isneginf(got_l[:, r0:r1]), ~fin)
            el = np.abs(got_l[:, r0:r1][fin] - Lb[fin])
            tl = d.T[fin] + 2.0 ** -20 * np.abs(Lb[fin]) + 2.0 ** -20
            assert np.all(el <= tl), (b, float((el / tl).max()))


CTX = [1, 17, 128, 300, 1000, 777, 129, 40, 16, 0]
QL = [1, 17, 100, 64, 300, 777, 1, 39, 0, 0]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("splits", [1, 0, 3])
def test_ragged_chunks(causal, splits):
    a = make(CTX, QL, seed=40)
    o, lse, st = run(*a[:3], causal, a[3], splits=splits)
    assert st == 0
    check(*a[:3], causal, a[3], o, lse)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (6, 3), (9, 3), (24, 4), (14, 2), (16, 2), (16, 1), (40, 8), (33, 1),
                                    (128, 1)])
@pytest.mark.parametrize("splits", [1, 2])
def test_head_layouts(Hq, Hkv, splits):
    a = make([50, 400, 131], [50, 131, 3], Hq=Hq, Hkv=Hkv, seed=Hq)
    o, lse, st = run(*a[:3], True, a[3], splits=splits)
    assert st == 0
    check(*a[:3], True, a[3], o, lse)


@pytest.mark.parametrize("T", [1, 2, 4, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("splits", [0, 1, 5])
def test_few_new_tokens(T, splits):
    a = make([T, T + 1, 640, 1290, 2047], [T] * 5, seed=T)
    o, lse, st = run(*a[:3], True, a[3], splits=splits)
    assert st == 0
    check(*a[:3], True, a[3], o, lse)


def test_single_tokens_agree_with_the_decode():
    import flashattention_attention_attn_b200 as fa
    ctx = [1, 15, 16, 17, 200, 511, 3000]
    q, cu, c, scale = make(ctx, [1] * 7, seed=3)
    o, lse, st = run(q, cu, c, True, scale)
    check(q, cu, c, True, scale, o, lse)
    od = torch.empty_like(q, device="cuda")
    fa.paged_attn_decode_fp8(q.cuda(), c.k_cache.cuda(), c.v_cache.cuda(), c.block_table.cuda(), c.seq_lens.cuda(), 7, 32,
                             8, 128, 16, c.block_table.shape[1], 0, c.k_scale, c.v_scale, od)
    torch.cuda.synchronize()
    # each within its own tolerance of the exact result
    check(q, cu, c, True, scale, od.cpu(), None)


@pytest.mark.parametrize("B", [31, 32, 33, 70])
def test_many_sequences(B):
    g = np.random.default_rng(B)
    ctx = g.integers(0, 700, B).tolist()
    ql = [int(min(c, x)) for c, x in zip(ctx, g.integers(0, 130, B))]
    ctx[-1], ql[-1] = 600, 300
    a = make(ctx, ql, Hq=8, Hkv=2, seed=B)
    for splits in (1, 2):
        o, lse, st = run(*a[:3], True, a[3], splits=splits, pad=5)
        assert st == 0
        check(*a[:3], True, a[3], o, lse)


def test_more_queries_than_keys_and_no_keys():
    """Rows before the first key see nothing: o = 0, lse = -inf."""
    a = make([10, 0, 200, 1], [40, 7, 260, 300], seed=8)
    for causal in (True, False):
        for splits in (1, 2):
            o, lse, st = run(*a[:3], causal, a[3], splits=splits)
            assert st == 0
            check(*a[:3], causal, a[3], o, lse)


@pytest.mark.parametrize("ql", [[5, 300, 70, 16], [4, 1, 3, 4], [8, 7, 1, 2]])
def test_placement_and_garbage_past_the_end(ql):
    q, cu, c, scale = make([37, 300, 1000, 16], ql, seed=75)
    for splits in (1, 2):
        want = run(q, cu, c, True, scale, splits=splits)
        g = torch.Generator().manual_seed(9)
        perm = torch.randperm(c.k_cache.shape[0], generator=g)
        k2, v2, table = torch.empty_like(c.k_cache), torch.empty_like(c.v_cache), c.block_table.clone()
        k2[perm], v2[perm] = c.k_cache, c.v_cache
        table[table >= 0] = perm[table[table >= 0].long()].to(torch.int32)
        for i, L in enumerate(c.seq_lens.tolist()):  # NaN codes behind each end
            last = int(table[i, (L - 1) // 16])
            k2[last, L % 16 or 16:] = 0x7F
            v2[last, L % 16 or 16:] = 0xFF
        e = inputs.PagedInputsFp8(c.q, k2, v2, table, c.seq_lens, 16, c.k_scale, c.v_scale)
        got = run(q, cu, e, True, scale, splits=splits)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        again = run(q, cu, e, True, scale, splits=splits, lse=False)  # and without an lse buffer
        assert torch.equal(again[0], want[0])


@pytest.mark.parametrize("ql", [[40, 300, 3], [4, 2, 3], [8, 1, 5]])
def test_ids_outside_the_pool_and_lengths_past_the_row(ql):
    q, cu, c, scale = make([500, 300, 64], ql, seed=21, spare=40)
    pool = c.k_cache.shape[0] - 20  # the last blocks stay inside the allocation
    t = c.block_table.clone()
    t[0, 3], t[0, 30], t[1, 0], t[1, 18] = -1, pool + 3, pool, 1 << 30
    t[2, :4] = pool + 7  # nothing left of this sequence
    keep = (t < pool)
    t[~keep & (t < 1 << 29) & (t >= 0)] = pool + 5
    e = inputs.PagedInputsFp8(c.q, c.k_cache, c.v_cache, t, c.seq_lens, 16, c.k_scale, c.v_scale)
    for splits in (1, 3):
        o, lse, st = run(q, cu, e, True, scale, splits=splits, num_blocks=pool)
        assert st == 0x2
        check(q, cu, e, True, scale, o, lse, num_blocks=pool)
    # lengths outside the table row's capacity are clamped into it
    width = c.block_table.shape[1]
    full = c.block_table.clone()
    full[full < 0] = 0
    f = inputs.PagedInputsFp8(c.q, c.k_cache, c.v_cache, full, torch.tensor([width * 16 + 9, -4, 64], dtype=torch.int32), 16,
                              c.k_scale, c.v_scale)
    o, lse, st = run(q, cu, f, True, scale, splits=2)
    assert st == 0x4
    check(q, cu, f, True, scale, o, lse)


@pytest.mark.parametrize("T", [70, 3, 8])
@pytest.mark.parametrize("factor", [2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 40])
def test_any_size_of_query(factor, T):
    """Rows are scaled by powers of two inside; with the score scale undone outside the result is the same."""
    q, cu, c, scale = make([200, 90], [T, 1], Hq=8, Hkv=2, seed=5)
    base = run(q, cu, c, True, scale)
    big = run((q.float() * factor).to(torch.bfloat16), cu, c, True, scale / factor)
    assert torch.equal(big[0], base[0]) and torch.allclose(big[1], base[1], rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("ql", [[300, 2], [4, 3], [8, 5]])
def test_uneven_rows_and_rising_scores(ql):
    """One element far above the rest of its row, rows of zeros, and keys that grow along the sequence, so that the
    running maximum moves many times."""
    q, cu, c, scale = make([900, 700], ql, seed=6)
    q[::3, :, 5] *= 300.0
    q[1] = 0.0
    codes = torch.arange(16 * c.k_cache.shape[0]) % 100  # a code that rises through each block
    c.k_cache[..., 9] = codes.view(-1, 16, 1).to(torch.uint8)
    for splits in (1, 4):
        o, lse, st = run(q, cu, c, True, scale, splits=splits)
        assert st == 0
        check(q, cu, c, True, scale, o, lse)


@pytest.mark.parametrize("T", [300, 4, 8])
def test_nan_query_row_stays_alone(T):
    q, cu, c, scale = make([300], [T], Hq=8, Hkv=2, seed=31)
    want = run(q, cu, c, True, scale, splits=1)
    q2 = q.clone()
    q2[T // 3, 3, 7], q2[2 * T // 3, 1, 0] = float("nan"), float("inf")
    for splits in (1, 2):
        got = run(q2, cu, c, True, scale, splits=splits)
        hit = torch.zeros(T, 8, dtype=torch.bool)
        hit[T // 3, 3] = hit[2 * T // 3, 1] = True
        assert torch.isnan(got[0][hit]).all() and torch.isnan(got[1].t()[hit]).all()
        ref = want if splits == 1 else run(q, cu, c, True, scale, splits=2)
        assert torch.equal(got[0][~hit], ref[0][~hit]) and torch.equal(got[1].t()[~hit], ref[1].t()[~hit])


def test_long_cache_few_rows():
    a = make([20000], [8], seed=50)
    o, lse, st = run(*a[:3], False, a[3])
    assert st == 0
    check(*a[:3], False, a[3], o, lse)


@pytest.mark.parametrize("T", [2, 8, 40])
def test_most_of_the_sum_in_small_weights(T):
    """One key far above all others (an attention sink) before thousands whose weights are 2^-13 of its: together they
    outweigh it, so the small weights' bits decide the result."""
    S, Hkv = 16000, 1
    q, cu, c, _ = make([S], [T], Hq=4, Hkv=Hkv, seed=90, k_scale=1.0)
    q[:] = 1.0
    c.k_cache[:] = 0
    first = int(c.block_table[0, 0])
    c.k_cache[first, 0, 0, :72] = 0x38  # 72 ones: a score of 9
    rest = torch.randint(0, 3, c.k_cache.shape[:3], generator=torch.Generator().manual_seed(2)).to(torch.uint8)
    c.k_cache[..., 127] += rest * 8  # small spread among the others
    c.v_cache[:] = 0x38  # values of one: o is the sum of the rounded weights over the sum of the weights
    c.v_cache[first, 0] = 0
    for splits in (1, 4):
        o, lse, st = run(q, cu, c, False, 0.125 * 8, splits=splits)
        assert st == 0
        check(q, cu, c, False, 0.125 * 8, o, lse)


def test_two_streams_and_a_captured_call():
    import flashattention_attention_attn_b200 as fa
    a, b = make([900, 33], [6, 33], seed=60), make([400], [200], seed=61)
    want = [run(*x[:3], True, x[3]) for x in (a, b)]
    outs, graphs = [], []
    for x in (a, b):
        q, cu, c, scale = x
        t = [y.cuda() for y in (q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, cu)]
        o = torch.zeros_like(t[0])
        lse = torch.zeros(32, q.shape[0], device="cuda")

        def call(t=t, o=o, lse=lse, c=c, scale=scale, q=q, cu=cu):
            fa.paged_attn_prefill_fp8(*t, len(cu) - 1, 32, 8, 128, 16, c.block_table.shape[1],
                                      int((cu[1:] - cu[:-1]).max()), q.shape[0], True, scale, c.k_scale, c.v_scale, 0, o,
                                      lse)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, call))
        outs.append((o, lse))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o, lse in outs:
            o.zero_(), lse.zero_()
        torch.cuda.synchronize()
        for s, (g, call) in zip(streams, graphs):  # the two graphs at once, then the two calls at once
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, lse), w in zip(outs, want):
            assert torch.equal(o.cpu(), w[0]) and torch.equal(lse.cpu(), w[1])
        for s, (g, call) in zip(streams, graphs):
            with torch.cuda.stream(s):
                call()
        torch.cuda.synchronize()
        for (o, lse), w in zip(outs, want):
            assert torch.equal(o.cpu(), w[0]) and torch.equal(lse.cpu(), w[1])
    assert fa.attn_read_device_status(clear=True) == 0


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 1), (16, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_few_long_units_are_cut(causal, Hq, Hkv):
    """Long keys and few query blocks, where the automatic choice deals the keys
    out evenly: a unit lies on many stretches, others between them end on one."""
    ctx, ql = [20000, 0, 9000, 4001, 1, 130], [100, 0, 60, 33, 1, 40]
    q, cu, c, scale = make(ctx, ql, Hq=Hq, Hkv=Hkv, seed=90 + Hq)
    o, lse, st = run(q, cu, c, causal, scale, pad=4)
    assert st == 0
    check(q, cu, c, causal, scale, o, lse)
    # the result does not depend on where the blocks lie, nor on what lies behind the ends
    g = torch.Generator().manual_seed(9)
    perm = torch.randperm(c.k_cache.shape[0], generator=g)
    k2, v2, table = torch.empty_like(c.k_cache), torch.empty_like(c.v_cache), c.block_table.clone()
    k2[perm], v2[perm] = c.k_cache, c.v_cache
    table[table >= 0] = perm[table[table >= 0].long()].to(torch.int32)
    for i, L in enumerate(c.seq_lens.tolist()):
        if L % 16:
            last = int(table[i, (L - 1) // 16])
            k2[last, L % 16:] = 0x7F
            v2[last, L % 16:] = 0xFF
    e = inputs.PagedInputsFp8(c.q, k2, v2, table, c.seq_lens, 16, c.k_scale, c.v_scale)
    again = run(q, cu, e, causal, scale, lse=False)
    assert torch.equal(again[0], o)


def test_cut_units_with_ids_outside_the_pool_and_nan_rows():
    ctx, ql = [9000, 3000, 4000], [70, 40, 50]
    q, cu, c, scale = make(ctx, ql, Hq=8, Hkv=2, seed=31, spare=20)
    pool = c.k_cache.shape[0] - 20
    t = c.block_table.clone()
    t[0, 3], t[0, 300:330], t[1, 0] = -1, pool + 3, pool
    t[2, : 4000 // 16] = pool + 7  # nothing left of this sequence
    e = inputs.PagedInputsFp8(c.q, c.k_cache, c.v_cache, t, c.seq_lens, 16, c.k_scale, c.v_scale)
    o, lse, st = run(q, cu, e, True, scale, num_blocks=pool)
    assert st == 0x2
    check(q, cu, e, True, scale, o, lse, num_blocks=pool)
    x = q.clone()
    x[10, 3] = float("nan")
    o2, lse2, st = run(x, cu, e, True, scale, num_blocks=pool)
    assert torch.isnan(o2[10, 3]).all() and torch.isnan(lse2[3, 10])
    o2[10, 3], lse2[3, 10] = o[10, 3], lse[3, 10]
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("B", [385, 800])
def test_more_sequences_than_threads(B):
    g = np.random.default_rng(B)
    ctx = g.integers(0, 150, B).tolist()
    ql = [int(min(c, x)) for c, x in zip(ctx, g.integers(0, 14, B))]
    ctx[400 % B], ql[400 % B] = 2500, 90  # tables wide enough for the automatic choice
    a = make(ctx, ql, Hq=8, Hkv=2, seed=B)
    for splits in (0, 1, 2):
        o, lse, st = run(*a[:3], True, a[3], splits=splits, pad=3)
        assert st == 0
        check(*a[:3], True, a[3], o, lse)


def test_cut_units_on_two_streams_and_captured():
    import flashattention_attention_attn_b200 as fa
    jobs, want = [], []
    for seed, ctx, ql in ((62, [9000, 700], [50, 60]), (63, [6000], [40])):
        q, cu, c, scale = make(ctx, ql, Hq=8, Hkv=2, seed=seed)
        o, lse, _ = run(q, cu, c, True, scale)
        check(q, cu, c, True, scale, o, lse)
        want.append((o, lse))
        t = [y.cuda() for y in (q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, cu)]
        out = (torch.zeros_like(t[0]), torch.zeros(8, q.shape[0], device="cuda"))

        def call(t=t, out=out, c=c, scale=scale, q=q, cu=cu):
            fa.paged_attn_prefill_fp8(*t, len(cu) - 1, 8, 2, 128, 16, c.block_table.shape[1],
                                      int((cu[1:] - cu[:-1]).max()), q.shape[0], True, scale, c.k_scale, c.v_scale, 0, *out)

        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        jobs.append((g, call, out))
    streams = [torch.cuda.Stream() for _ in jobs]
    for use_graph in (True, False, True):
        for _, _, out in jobs:
            out[0].zero_(), out[1].zero_()
        torch.cuda.synchronize()
        for s, (g, call, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                g.replay() if use_graph else call()
        torch.cuda.synchronize()
        for (_, _, out), w in zip(jobs, want):
            assert torch.equal(out[0].cpu(), w[0]) and torch.equal(out[1].cpu(), w[1])
    assert fa.attn_read_device_status(clear=True) == 0


@pytest.mark.parametrize("splits", [0, 1, 2])
def test_more_units_than_sms_on_two_streams_and_captured(splits):
    """Hundreds of units, which running CTAs take over from the grid, in two
    calls at once, eager and replayed: the same bits as one call alone."""
    import flashattention_attention_attn_b200 as fa
    jobs = []
    for seed, B in ((64, 41), (65, 23)):
        g = np.random.default_rng(seed)
        ctx = g.integers(0, 2200, B).tolist()
        ql = [int(min(c, x)) for c, x in zip(ctx, g.integers(0, 200, B))]
        ctx[3], ql[3] = 2300, 200
        q, cu, c, scale = make(ctx, ql, seed=seed)
        want = run(q, cu, c, True, scale, splits=splits)
        check(q, cu, c, True, scale, *want[:2])
        t = [y.cuda() for y in (q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, cu)]
        out = (torch.zeros_like(t[0]), torch.zeros(32, q.shape[0], device="cuda"))

        def call(t=t, out=out, c=c, scale=scale, q=q, cu=cu, B=B):
            fa.paged_attn_prefill_fp8(*t, B, 32, 8, 128, 16, c.block_table.shape[1], int((cu[1:] - cu[:-1]).max()),
                                      q.shape[0], True, scale, c.k_scale, c.v_scale, splits, *out)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        jobs.append((graph, call, out, want))
    streams = [torch.cuda.Stream() for _ in jobs]
    for use_graph in (True, False, True, False):
        for _, _, out, _ in jobs:
            out[0].zero_(), out[1].zero_()
        torch.cuda.synchronize()
        for s, (graph, call, _, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                graph.replay() if use_graph else call()
        torch.cuda.synchronize()
        for _, _, out, want in jobs:
            assert torch.equal(out[0].cpu(), want[0]) and torch.equal(out[1].cpu(), want[1])
    assert fa.attn_read_device_status(clear=True) == 0
