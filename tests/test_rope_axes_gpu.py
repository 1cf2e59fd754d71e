"""rope_axes_fwd / _bwd and the cache-writing forms against the fp64 oracle.

Tolerance of a bf16 result y: half a step, 2^-8 |y|, and the fp32 rotation
a c - b s before it: c and s within 2^-22, two products and a sum of relative
error 2^-24 each, together under 2^-21 (|a| + |b|).  An e4m3 code of x: half a
step, max(2^-4 |x|, 2^-10), and the same fp32 error over the scale, with the
quotient's own rounding, 2^-24 |x|."""

import numpy as np
import pytest
import torch

from oracle import fp64_attention as orc
from oracle import paged_step as ps

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def status():
    import flashattention_attention_attn_b200 as fa
    return fa.attn_read_device_status(clear=True)


def rope_inputs(seed, n, Hq, Hkv, d, rot, axes, far=4096):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(n, (Hq + 2 * Hkv) * d, generator=g).to(BF16)
    pos = torch.randint(0, far, (axes, n), generator=g, dtype=torch.int32)
    half = rot // 2
    f = (500000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()
    axis = bytes(int(a) for a in torch.randint(0, axes, (half,), generator=g))
    return qkv, pos, f, axis


def heads(x, H, d):
    return f64(x).reshape(x.shape[0], H, d)


def pair_sum(x, rot, adjacent):
    """|a| + |b| of every element's pair."""
    a = np.abs(x)
    out = a.copy()
    h = rot // 2
    if adjacent:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = s, s
    else:
        s = a[..., :h] + a[..., h:rot]
        out[..., :h], out[..., h:rot] = s, s
    return out


def close(got, want, x, rot, adjacent):
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * pair_sum(x, rot, adjacent)
    err = np.abs(got - want)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())
    assert np.array_equal(got[..., rot:], x[..., rot:])  # what is not rotated is copied


def oracle(x, pos, f, axis, adjacent, sign=1.0):
    return ps.rope_axes(x, pos.numpy(), f64(f), axis, adjacent, sign)


CASES = [  # n, Hq, Hkv, d, rot, axes, adjacent, fused
    (1, 32, 8, 128, 128, 1, False, True),
    (7, 32, 8, 128, 128, 3, False, True),
    (129, 24, 4, 128, 64, 2, True, False),
    (700, 5, 5, 64, 64, 3, False, False),
    (1301, 7, 1, 64, 32, 2, True, True),
    (2500, 2, 2, 128, 112, 4, False, True),
    (3, 8, 2, 128, 16, 1, True, False),
    (5, 3, 1, 64, 0, 1, False, False),
]


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,axes,adjacent,fused", CASES)
def test_rotation_and_gradient(n, Hq, Hkv, d, rot, axes, adjacent, fused, bwd):
    import flashattention_attention_attn_b200 as fa
    qkv, pos, f, axis = rope_inputs(n + rot, n, Hq, Hkv, d, rot, axes)
    dev = qkv.cuda()
    q, k = dev[:, :Hq * d], dev[:, Hq * d:(Hq + Hkv) * d]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    qo = torch.full((n + 1, Hq * d + 8), float("nan"), device="cuda", dtype=BF16)  # rows with a gap, one row too many
    ko = torch.full((n + 1, Hkv, d), float("nan"), device="cuda", dtype=BF16)
    call = fa.rope_axes_bwd if bwd else fa.rope_axes_fwd
    call(q, k, pos.cuda(), f.cuda(), axis, n, Hq, Hkv, d, rot, axes, n, q.stride(0), k.stride(0), adjacent, qo, ko,
         Hq * d + 8, Hkv * d)
    torch.cuda.synchronize()
    assert status() == 0
    sign = -1.0 if bwd else 1.0
    xq, xk = heads(q, Hq, d), heads(k, Hkv, d)
    close(heads(qo[:n, :Hq * d], Hq, d), oracle(xq, pos, f, axis, adjacent, sign), xq, rot, adjacent)
    close(f64(ko[:n]), oracle(xk, pos, f, axis, adjacent, sign), xk, rot, adjacent)
    assert torch.isnan(qo[n]).all() and torch.isnan(qo[:, Hq * d:]).all() and torch.isnan(ko[n]).all()
    assert torch.equal(dev.cpu(), qkv)


def test_far_positions_keep_their_angle():
    import flashattention_attention_attn_b200 as fa
    n, d = 64, 128
    qkv, _, f, _ = rope_inputs(3, n, 2, 1, d, d, 1)
    pos = (2 ** 31 - 1 - 977 * torch.arange(n, dtype=torch.int64)).to(torch.int32)[None]
    pos[0, ::2] = 1048575 - torch.arange(n // 2, dtype=torch.int32)
    pos[0, 1] = -131072
    q = qkv[:, :2 * d].contiguous().cuda()
    k = qkv[:, 2 * d:3 * d].contiguous().cuda()
    x, xk = heads(q, 2, d), heads(k, 1, d)
    fa.rope_axes_fwd(q, k, pos.cuda(), f.cuda(), None, n, 2, 1, d, d, 1, 0, 2 * d, d, False, q, k, 2 * d, d)  # in place
    torch.cuda.synchronize()
    close(heads(q, 2, d), oracle(x, pos, f, bytes(d // 2), False), x, d, False)
    close(heads(k, 1, d), oracle(xk, pos, f, bytes(d // 2), False), xk, d, False)


def test_one_row_of_positions_for_all_axes_and_a_head_kind_left_out():
    import flashattention_attention_attn_b200 as fa
    n, Hq, d = 33, 6, 64
    qkv, pos, f, axis = rope_inputs(8, n, Hq, 1, d, d, 3)
    q = qkv[:, :Hq * d].contiguous().cuda()
    out = torch.empty_like(q)
    fa.rope_axes_fwd(q, None, pos.cuda(), f.cuda(), axis, n, Hq, 0, d, d, 3, 0, Hq * d, 0, False, out, None, Hq * d, 0)
    k_out = torch.empty_like(q)
    fa.rope_axes_fwd(None, q, pos.cuda(), f.cuda(), axis, n, 0, Hq, d, d, 3, 0, 0, Hq * d, False, None, k_out, 0, Hq * d)
    torch.cuda.synchronize()
    x = heads(q, Hq, d)
    close(heads(out, Hq, d), oracle(x, pos[:1].expand(3, n), f, axis, False), x, d, False)
    assert torch.equal(out, k_out)


def test_gradient_against_differences():
    """d <g, rope(x)> / dx by central differences of the oracle, which is linear in x: exact up to rounding."""
    import flashattention_attention_attn_b200 as fa
    n, H, d = 4, 2, 64
    qkv, pos, f, axis = rope_inputs(12, n, H, 1, d, d, 2)
    g = qkv[:, :H * d].contiguous()
    dq = torch.empty_like(g, device="cuda")
    fa.rope_axes_bwd(g.cuda(), None, pos.cuda(), f.cuda(), axis, n, H, 0, d, d, 2, n, H * d, 0, True, dq, None, H * d, 0)
    gg = heads(g, H, d)
    x = np.random.default_rng(0).standard_normal((n, H, d))
    want = np.zeros_like(x)
    for h in range(H):
        for e in range(d):
            hi, lo = x.copy(), x.copy()
            hi[:, h, e] += 0.5
            lo[:, h, e] -= 0.5
            delta = oracle(hi, pos, f, axis, True) - oracle(lo, pos, f, axis, True)
            want[:, h, e] = (gg * delta).sum((1, 2))
    close(heads(dq, H, d), want, gg, d, True)


def append_inputs(seed, n, Hq, Hkv, d, rot, axes, pool):
    qkv, pos, f, axis = rope_inputs(seed, n, Hq, Hkv, d, rot, axes)
    g = torch.Generator().manual_seed(seed + 1)
    slots = torch.randperm(pool * 16, generator=g)[:n].to(torch.int32)
    return qkv, pos, f, axis, slots


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,axes,adjacent,fused", CASES)
def test_append(n, Hq, Hkv, d, rot, axes, adjacent, fused, fp8):
    import flashattention_attention_attn_b200 as fa
    if fp8 and d != 128:
        d, rot = 128, rot * 2
    pool = n // 16 + 3
    qkv, pos, f, axis, slots = append_inputs(n + 3 * rot, n, Hq, Hkv, d, rot, axes, pool)
    if n > 2:
        slots[1] = -1  # padding in the middle
    if n > 700:
        slots[-3:] = -5
    ks, vs = 0.0213, 0.31
    dev = qkv.cuda()
    q, k, v = dev[:, :Hq * d], dev[:, Hq * d:(Hq + Hkv) * d], dev[:, (Hq + Hkv) * d:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qo = torch.full((n + 1, Hq, d), float("nan"), device="cuda", dtype=BF16)
    if fp8:
        kc, vc = (torch.randint(0, 256, (pool, 16, Hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    else:
        kc, vc = (torch.randn(pool, 16, Hkv, d, device="cuda").to(BF16) for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    args = (q, k, v, pos.cuda(), f.cuda(), axis, slots.cuda(), n, Hq, Hkv, d, rot, axes, n, q.stride(0), k.stride(0),
            v.stride(0), adjacent, 16, pool)
    if fp8:
        fa.rope_axes_paged_append_fp8(*args, ks, vs, qo, kc, vc)
    else:
        fa.rope_axes_paged_append(*args, qo, kc, vc)
    torch.cuda.synchronize()
    assert status() == 0
    xq, xk, xv = heads(q, Hq, d), heads(k, Hkv, d), heads(v, Hkv, d)
    close(f64(qo[:n]), oracle(xq, pos, f, axis, adjacent), xq, rot, adjacent)
    assert torch.isnan(qo[n]).all()
    rk = oracle(xk, pos, f, axis, adjacent)
    used = np.zeros(pool * 16, bool)
    real = slots.numpy() >= 0
    used[slots.numpy()[real]] = True
    at = slots.long()[torch.from_numpy(real)].cuda()
    for cache, before in ((kc, k0), (vc, v0)):  # every other slot as it was
        assert torch.equal(cache.view(pool * 16, -1).cpu()[~used], before.view(pool * 16, -1).cpu()[~used])
    gk, gv = kc.view(pool * 16, Hkv, d)[at], vc.view(pool * 16, Hkv, d)[at]
    if not fp8:
        close(f64(gk), rk[real], xk[real], rot, adjacent)
        assert torch.equal(gv, v.reshape(n, Hkv, d)[torch.from_numpy(real).cuda()])
        return
    for codes, x, scale, pairs in ((gk, rk[real], ks, pair_sum(xk[real], rot, adjacent)), (gv, xv[real], vs, 0.0)):
        scale = float(np.float32(scale))
        x = np.clip(x / scale, -448, 448)
        tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) + 2.0 ** -21 * pairs / scale + 2.0 ** -23 * np.abs(x)
        assert np.all(np.abs(orc.decode_e4m3(codes.cpu().numpy()) - x) <= tol)


def test_fp8_codes_are_the_nearest_saturated_ones():
    """Unrotated (position 0) values straight from the definition: ties, overflow, infinities, NaN, zeros."""
    import flashattention_attention_attn_b200 as fa
    v = ps.e4m3_values()
    x = np.concatenate([v, -v, (v[1:] + v[:-1]) / 2, [449, 460, 500, 1e6, -1e30, 0.0, -0.0, 2.0 ** -11, 2.0 ** -10]])
    x = torch.from_numpy(np.resize(x, 4 * 128)).to(BF16)
    x[7], x[8], x[9] = float("inf"), float("-inf"), float("nan")
    x = x.view(4, 128).cuda()
    for scale in (1.0, 0.25):
        kc, vc = torch.zeros(1, 16, 1, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, 16, 1, 128, dtype=torch.uint8,
                                                                                         device="cuda")
        fa.rope_axes_paged_append_fp8(None, x, x, torch.zeros(4, dtype=torch.int32, device="cuda"),
                                      torch.ones(64, device="cuda"), None, torch.arange(4, dtype=torch.int32, device="cuda"),
                                      4, 0, 1, 128, 128, 1, 4, 0, 128, 128, False, 16, 1, scale, scale, None, kc, vc)
        torch.cuda.synchronize()
        with np.errstate(over="ignore"):
            y = f64(x) / scale
        want = ps.nearest_e4m3(np.where(np.isnan(y), 0, y))
        nan = np.isnan(y)
        got = vc[0, :4, 0].cpu().numpy()
        assert np.array_equal(got[~nan], want[~nan]) and np.all((got[nan] & 0x7F) == 0x7F)


def test_slots_past_the_pool_are_dropped_and_flagged():
    import flashattention_attention_attn_b200 as fa
    n, d = 6, 64
    qkv, pos, f, axis, _ = append_inputs(4, n, 2, 1, d, d, 1, 4)
    slots = torch.tensor([0, 31, 32, 63, 2**31 - 1, -2**31], dtype=torch.int32)  # the pool given below has two blocks
    dev = qkv.cuda()
    kc = torch.zeros(4, 16, 1, d, device="cuda", dtype=BF16)
    vc, qo = torch.zeros_like(kc), torch.zeros(n, 2, d, device="cuda", dtype=BF16)
    fa.rope_axes_paged_append(dev[:, :2 * d], dev[:, 2 * d:3 * d], dev[:, 3 * d:], pos.cuda(), f.cuda(), axis,
                              slots.cuda(), n, 2, 1, d, d, 1, n, 4 * d, 4 * d, 4 * d, False, 16, 2, qo, kc, vc)
    torch.cuda.synchronize()
    assert status() == 0x2
    assert vc.view(64, d).abs().sum(-1).nonzero().flatten().tolist() == [0, 31]
    assert torch.all(qo.abs().sum(-1) > 0)
