"""The serving step as it is used: plan, cache write, attention, step after step
over one cache, against the fp64 oracle of the whole; the torch ops of it."""

import numpy as np
import pytest
import torch

from oracle import fp64_attention as orc
from oracle import paged_step as ps

BF16 = torch.bfloat16
HQ, HKV, D, ROT = 16, 4, 128, 96


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Server:
    """Requests over one paged cache, and the same history kept in fp64."""

    def __init__(self, B, fp8, seed):
        import flashattention_attention_attn_b200 as fa
        import flashattention_attention_attn_b200.torch_ops  # noqa: F401
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.fp8, self.pool, self.width = B, fp8, 260, 40
        self.axes = fa.rope_axis_map([12, 20, 16], interleaved=True)
        self.f = (10000.0 ** (-torch.arange(ROT // 2, dtype=torch.float64) / (ROT // 2))).float()
        self.free = torch.randperm(self.pool, generator=self.g).to(torch.int32)
        self.cached = torch.zeros(B, dtype=torch.int32)
        self.table = torch.full((B, self.width), -1, dtype=torch.int32, device="cuda")
        dt = torch.uint8 if fp8 else BF16
        self.kc = torch.zeros(self.pool, 16, HKV, D, dtype=dt, device="cuda")
        self.vc = torch.zeros_like(self.kc)
        self.ks, self.vs = (0.019, 0.023) if fp8 else (1.0, 1.0)
        self.hist = [([], []) for _ in range(B)]  # fp64 k, v rows as the cache holds them

    def step(self, new):
        ops = torch.ops.fa_b200
        B, total = self.B, sum(new)
        pad = 3
        new_t = torch.tensor(new, dtype=torch.int32)
        want = ps.plan_step(self.cached.tolist(), new, self.free.tolist(), None, self.table.cpu().numpy(), total + pad)
        lens, cu, slots, pos, taken = ops.paged_cache_plan(self.table, self.cached.cuda(), new_t.cuda(), self.free.cuda(),
                                                           None, total + pad)
        for k, v in (("block_table", self.table), ("seq_lens", lens), ("cu_seqlens_q", cu), ("slot_map", slots),
                     ("positions", pos), ("blocks_taken", taken)):
            assert np.array_equal(v.cpu().numpy(), want[k]), k
        qkv = torch.randn(total + pad, (HQ + 2 * HKV) * D, generator=self.g).to(BF16).cuda()
        q = qkv[:, :HQ * D].view(-1, HQ, D)
        k = qkv[:, HQ * D:(HQ + HKV) * D].view(-1, HKV, D)
        v = qkv[:, (HQ + HKV) * D:].view(-1, HKV, D)
        axes = torch.stack([pos, pos // 3, pos * 2])  # three axes made from the plan's positions
        args = (q, k, v, axes, self.f.cuda(), list(self.axes), slots, False, self.kc, self.vc)
        scale = 1 / np.sqrt(D)
        mx = max(new)
        if self.fp8:
            qr = ops.rope_axes_paged_append_fp8(*args, self.ks, self.vs)
            o, lse = ops.paged_attn_prefill_fp8(qr, self.kc, self.vc, self.table, lens, cu, mx, True, scale, self.ks,
                                                self.vs, 0)
        else:
            qr = ops.rope_axes_paged_append(*args)
            o, lse = ops.paged_attn_prefill(qr, self.kc, self.vc, self.table, lens, cu, mx, True, scale)
        if mx == 1 and min(new) == 1:  # a decode step: the decode over the same cache agrees
            qd = qr[:B].contiguous()
            od = (ops.paged_attn_decode_fp8(qd, self.kc, self.vc, self.table, lens, 0, self.ks, self.vs) if self.fp8
                  else ops.paged_attn_decode(qd, self.kc, self.vc, self.table, lens, 0))
            assert np.abs(f64(od) - f64(o[:B])).max() <= 2e-2
        torch.cuda.synchronize()
        # the same in fp64, from the rotated rows rounded to what the cache holds
        axes_n = axes.cpu().numpy()
        rk = ps.rope_axes(f64(k), axes_n, f64(self.f), list(self.axes), False)
        rv = f64(v)
        rq = ps.rope_axes(f64(q), axes_n, f64(self.f), list(self.axes), False)
        # (the attention is checked on the values stored: a rounding may go either way at a border)
        held_k = orc.decode_e4m3(self.kc.cpu().numpy()) * np.float64(np.float32(self.ks)) if self.fp8 else f64(self.kc)
        held_v = orc.decode_e4m3(self.vc.cpu().numpy()) * np.float64(np.float32(self.vs)) if self.fp8 else f64(self.vc)
        at = slots.cpu().numpy()[:total]
        step = 2.0 ** -4 if self.fp8 else 2.0 ** -8  # half a step of the cache's type, relative
        for held, x, s in ((held_k, rk, self.ks), (held_v, rv, self.vs)):
            got = held.reshape(-1, HKV, D)[at]
            assert np.all(np.abs(got - x[:total]) <= step * np.abs(x[:total]) + (2.0 ** -10 * s if self.fp8 else 0) + 1e-5)
        assert np.all(np.abs(f64(qr[:total]) - rq[:total]) <= 2.0 ** -8 * np.abs(rq[:total]) + 1e-5)
        t = 0
        for b, n in enumerate(new):
            for i in range(n):
                slot = int(at[t])
                self.hist[b][0].append(held_k[slot // 16, slot % 16])
                self.hist[b][1].append(held_v[slot // 16, slot % 16])
                t += 1
            K, V = np.array(self.hist[b][0]), np.array(self.hist[b][1])
            assert len(K) == int(lens[b])
            if n:
                O, L = orc.attention(f64(qr[t - n:t])[None], K[None], V[None], scale, True)
                assert np.abs(f64(o[t - n:t]) - O[0]).max() <= 2e-2
                assert np.abs(f64(lse[:, t - n:t]) - L[0]).max() <= 1e-3
        self.cached = lens.cpu()
        self.free = self.free[int(taken):]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_a_server_runs_prompts_chunks_drafts_and_decode_steps(fp8):
    import flashattention_attention_attn_b200 as fa
    s = Server(5, fp8, seed=3)
    for new in ([90, 1, 33, 0, 17], [40, 1, 200, 5, 0], [4, 4, 4, 4, 4], [1, 1, 1, 1, 1], [8, 0, 3, 8, 1], [1, 1, 1, 1, 1]):
        s.step(new)
    assert fa.attn_read_device_status(clear=True) == 0


@pytest.mark.gpu
def test_a_captured_step_follows_new_lengths():
    """plan, FP8 cache write and attention in one graph, replayed for other lengths, against the calls one by one."""
    import flashattention_attention_attn_b200 as fa
    import flashattention_attention_attn_b200.torch_ops  # noqa: F401
    B, width, pool, cap, T = 6, 30, 200, 48, 8
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    cached, new, free = torch.zeros(B, **i32), torch.ones(B, **i32), torch.arange(pool, **i32)
    table = torch.full((B, width), -1, **i32)
    kc = torch.randint(0, 120, (pool, 16, HKV, D), dtype=torch.uint8, device="cuda", generator=g)
    vc = torch.randint(0, 120, (pool, 16, HKV, D), dtype=torch.uint8, device="cuda", generator=g)
    q = torch.randn(cap, HQ, D, device="cuda", generator=g).to(BF16)
    k, v = (torch.randn(cap, HKV, D, device="cuda", generator=g).to(BF16) for _ in range(2))
    f = torch.rand(D // 2, device="cuda", generator=g)
    out = [torch.zeros(n, **i32) for n in (B, B + 1, cap, cap, 1)]
    qr, o, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(HQ, cap, device="cuda")

    def call():
        lens, cu, slots, pos, taken = out
        fa.paged_cache_plan(cached, new, free, None, B, pool, 16, width, cap, table, lens, cu, slots, pos, taken)
        fa.rope_axes_paged_append_fp8(q, k, v, pos, f, None, slots, cap, HQ, HKV, D, D, 1, cap, HQ * D, HKV * D, HKV * D,
                                      True, 16, pool, 0.02, 0.03, qr, kc, vc)
        fa.paged_attn_prefill_fp8_checked(qr, kc, vc, table, lens, cu, B, HQ, HKV, D, 16, width, pool, T, cap, True, 0.09,
                                          0.02, 0.03, 0, o, lse)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    rng = np.random.default_rng(0)
    k0, v0 = kc.clone(), vc.clone()
    for _ in range(4):
        c, n = rng.integers(0, 400, B), rng.integers(0, T + 1, B)
        t = np.full((B, width), -1)
        ids = rng.permutation(pool)
        at = 0
        for b in range(B):
            t[b, :-(-c[b] // 16)] = ids[at:at - (-c[b] // 16)]
            at += -(-c[b] // 16)
        rest = ids[at:]
        results = []
        for run in (graph.replay, call):
            for dst, src in ((cached, c), (new, n), (table, t), (free, np.resize(rest, pool))):
                dst.copy_(torch.tensor(src, **i32))
            kc.copy_(k0), vc.copy_(v0), o.zero_(), lse.zero_()
            run()
            torch.cuda.synchronize()
            results.append([x.clone() for x in (*out, table, qr, kc, vc, o, lse)])
        for a, b in zip(*results):
            assert torch.equal(a, b)
        total = int(n.sum())
        assert torch.all(results[0][9][total:] == 0) and torch.all(results[0][9][:total].float().abs().sum(-1) > 0)
    assert fa.attn_read_device_status(clear=True) == 0


@pytest.mark.gpu
def test_rope_op_trains():
    """Gradients of q and k through the op, eager, strided, with one output unused, and compiled."""
    import flashattention_attention_attn_b200.torch_ops  # noqa: F401
    n, Hq, Hkv, d = 37, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(n, (Hq + Hkv) * d, generator=g).to(BF16).cuda().requires_grad_()
    pos = torch.randint(0, 3000, (2, n), generator=g, dtype=torch.int32).cuda()
    f = torch.rand(d // 2, generator=g).cuda()
    axis = [i % 2 for i in range(d // 2)]
    gq, gk = (torch.randn(n, h, d, generator=g).to(BF16).cuda() for h in (Hq, Hkv))

    def step(x, both=True):
        q, k = x[:, :Hq * d].view(n, Hq, d), x[:, Hq * d:].view(n, Hkv, d)
        a, b = torch.ops.fa_b200.rope_axes(q, k, pos, f, axis, True)
        return (a * gq).sum() + ((b * gk).sum() if both else 0.0)

    for both in (True, False):
        want_q = ps.rope_axes(f64(gq), pos.cpu().numpy(), f64(f), axis, True, sign=-1.0)
        want_k = ps.rope_axes(f64(gk) * both, pos.cpu().numpy(), f64(f), axis, True, sign=-1.0)
        want = np.concatenate([want_q.reshape(n, -1), want_k.reshape(n, -1)], 1)
        grads = [torch.autograd.grad(step(qkv, both), qkv)[0]]
        if both:
            grads.append(torch.autograd.grad(torch.compile(step, fullgraph=True, backend="aot_eager")(qkv), qkv)[0])
        for got in grads:
            assert np.all(np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)


@pytest.mark.gpu
def test_rope_op_takes_an_expanded_gradient_and_a_captured_step():
    """A gradient whose rows share their memory; forward and backward captured
    while an eager graph of the same leaves lives, made on the stream of the
    capture (made on the default stream it stops the capture of any torch
    operator's backward, x * 2 as well)."""
    import flashattention_attention_attn_b200.torch_ops  # noqa: F401
    n, H, d = 29, 3, 64
    g = torch.Generator().manual_seed(6)
    q, k = (torch.randn(n, H, d, generator=g).to(BF16).cuda().requires_grad_() for _ in range(2))
    pos = torch.randint(0, 3000, (1, n), generator=g, dtype=torch.int32).cuda()
    f = torch.rand(d // 2, generator=g).cuda()
    row = torch.randn(H, d, generator=g).to(BF16).cuda()
    want = ps.rope_axes(f64(row.expand(n, H, d)), pos.cpu().numpy(), f64(f), [0] * (d // 2), False, sign=-1.0)

    def grads():
        a, b = torch.ops.fa_b200.rope_axes(q, k, pos, f, [], False)
        return torch.autograd.grad((a, b), (q, k), (row.expand(n, H, d), row.expand(n, H, d)))

    for got in grads():
        assert np.all(np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
    q, k = (x.detach().requires_grad_() for x in (q, k))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        alive = sum(x.sum() for x in torch.ops.fa_b200.rope_axes(q, k, pos, f, [], False))
        grads()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = grads()
    with torch.no_grad():
        row.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    for got in captured:
        assert np.all(np.abs(f64(got) - 2 * want) <= 2.0 ** -7 * np.abs(want) + 2e-5)
    assert all(torch.isfinite(x).all() for x in torch.autograd.grad(alive, (q, k)))


@pytest.mark.gpu
def test_tensors_off_the_current_device_are_refused():
    import flashattention_attention_attn_b200 as fa
    x = torch.zeros(4, 128, dtype=BF16, device="cuda")
    host = torch.zeros(4, dtype=torch.int32)
    f = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        fa.rope_axes_fwd(x, x, host, f, None, 4, 1, 1, 128, 128, 1, 4, 128, 128, False, x, x, 128, 128)
    with pytest.raises(ValueError):
        fa.paged_cache_plan(host, host, host, None, 4, 4, 16, 2, 4, host, host, host, host, host, host)


@pytest.mark.gpu
def test_ops_take_strided_rows_and_refuse_other_types():
    import flashattention_attention_attn_b200.torch_ops  # noqa: F401
    ops = torch.ops.fa_b200
    g = torch.Generator().manual_seed(2)
    x = torch.randn(9, 6, 64, generator=g).to(BF16).cuda()
    f, pos = torch.rand(32, generator=g).cuda(), torch.arange(9, dtype=torch.int32, device="cuda")[None]
    want = ops.rope_axes(x, x[:, :2].contiguous(), pos, f, [], False)
    for y in (x.transpose(0, 1).contiguous().transpose(0, 1),               # heads apart
              torch.cat([x, x], 2)[..., :64], torch.cat([x, x], 1)[:, :6]):  # gaps within and between rows
        got = ops.rope_axes(y, y[:, :2], pos.t().contiguous().t(), f, [], False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError):
        ops.rope_axes(x.float(), x, pos, f, [], False)
    with pytest.raises(ValueError):
        ops.rope_axes(x, x, pos.long(), f, [], False)
    kc = torch.zeros(4, 16, 6, 64, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        ops.rope_axes_paged_append(x, x, x, pos, f, [], pos[0], False, kc.transpose(0, 1), kc)
    with pytest.raises(ValueError):
        ops.paged_attn_prefill_fp8(x, kc, kc, pos, pos[0], pos[0], 1, True, 1.0, 1.0, 1.0, 0)


def test_fake_shapes():
    import flashattention_attention_attn_b200.torch_ops  # noqa: F401
    ops = torch.ops.fa_b200
    with torch._subclasses.FakeTensorMode():
        i32 = dict(dtype=torch.int32)
        table = torch.empty(5, 9, **i32)
        out = ops.paged_cache_plan(table, torch.empty(5, **i32), torch.empty(5, **i32), torch.empty(7, **i32), None, 31)
        assert [tuple(x.shape) for x in out] == [(5,), (6,), (31,), (31,), (1,)]
        q, k = torch.empty(31, 8, 128, dtype=BF16), torch.empty(31, 2, 128, dtype=BF16)
        pos, f = torch.empty(3, 31, **i32), torch.empty(64)
        a, b = ops.rope_axes(q, k, pos, f, [0] * 64, False)
        assert a.shape == q.shape and b.shape == k.shape
        kc = torch.empty(9, 16, 2, 128, dtype=BF16)
        assert ops.rope_axes_paged_append(q, k, k, pos, f, [], out[2], False, kc, kc.clone()).shape == q.shape
        k8 = torch.empty(9, 16, 2, 128, dtype=torch.uint8)
        assert ops.rope_axes_paged_append_fp8(q, k, k, pos, f, [], out[2], False, k8, k8.clone(), 1.0, 1.0).shape == q.shape
        o, lse = ops.paged_attn_prefill_fp8(q, k8, k8, table, out[0], out[1], 8, True, 0.1, 1.0, 1.0, 0)
        assert o.shape == q.shape and lse.shape == (8, 31) and lse.dtype == torch.float32
