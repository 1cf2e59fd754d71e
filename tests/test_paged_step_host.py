"""The serving step around the paged cache, without a GPU: refusals of its
entry points (status codes as documented in attn.h), the axis map, and pins of
its oracle."""

import ctypes

import numpy as np
import pytest
import torch

from flashattention_attention_attn_b200 import build
from oracle import fp64_attention as orc
from oracle import paged_step as ps

OK, INVALID, UNSUPPORTED = 0, -1, -2
P = 1 << 20  # an aligned address that the host checks never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    from flashattention_attention_attn_b200 import _binding
    return _binding.library()


def _without_device(rc):
    """Status of a valid call: a machine without a device answers with a CUDA error, never with success."""
    return rc == -3 or (rc == OK and torch.cuda.is_available())


def _plan(lib, ptrs=(P,) * 10, B=4, num_free=8, bs=16, maxb=8, max_tokens=64):
    c, n, f, po, t, sl, cu, sm, pos, bt = ptrs
    return lib.paged_cache_plan(c, n, f, po, B, num_free, bs, maxb, max_tokens, t, sl, cu, sm, pos, bt, None)


def _p(i, v, n):
    return tuple(v if j == i else P for j in range(n))


@pytest.mark.parametrize("kw,expect", [
    *[(dict(ptrs=_p(i, None, 10)), INVALID) for i in (0, 1, 2, 4, 5, 6, 7, 8, 9)],
    (dict(B=-1), INVALID),
    (dict(num_free=-1), INVALID),
    (dict(maxb=0), INVALID),
    (dict(max_tokens=-1), INVALID),
    (dict(bs=0), INVALID),
    (dict(bs=32), UNSUPPORTED),
    (dict(maxb=1 << 27), UNSUPPORTED),
    *[(dict(ptrs=_p(i, P + 2, 10)), UNSUPPORTED) for i in range(10)],
])
def test_plan_refusals(lib, kw, expect):
    assert _plan(lib, **kw) == expect


def _rope(lib, fn="rope_axes_fwd", ptrs=(P,) * 6, axis=None, n=4, Hq=8, Hkv=2, d=128, rot=128, axes=1, ps_=4, qs=1024,
          ks=256, qos=1024, kos=256):
    q, k, pos, f, qo, ko = ptrs
    return getattr(lib, fn)(q, k, pos, f, axis, n, Hq, Hkv, d, rot, axes, ps_, qs, ks, 0, qo, ko, qos, kos, None)


@pytest.mark.parametrize("fn", ["rope_axes_fwd", "rope_axes_bwd"])
@pytest.mark.parametrize("kw,expect", [
    *[(dict(ptrs=_p(i, None, 6)), INVALID) for i in range(6)],
    (dict(n=-1), INVALID),
    (dict(Hq=-1), INVALID),
    (dict(d=0), INVALID),
    (dict(axes=0), INVALID),
    (dict(rot=144), INVALID),                       # more than the head
    (dict(rot=-16), INVALID),
    (dict(ps_=-4), INVALID),
    (dict(axis=bytes([0] * 63 + [1]), axes=1), INVALID),
    (dict(qs=1016), INVALID),                       # rows overlap
    (dict(kos=248), INVALID),
    (dict(d=96, rot=96), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED),
    (dict(qs=1028), UNSUPPORTED),                   # row not 16-byte aligned
    (dict(ptrs=_p(0, P + 8, 6)), UNSUPPORTED),
    (dict(ptrs=_p(5, P + 8, 6)), UNSUPPORTED),
    (dict(ptrs=_p(2, P + 2, 6)), UNSUPPORTED),
    (dict(n=0), OK),
    (dict(n=0, ptrs=(None,) * 6), OK),
    (dict(Hq=0, Hkv=0, ptrs=(None,) * 6), OK),
])
def test_rope_refusals(lib, fn, kw, expect):
    assert _rope(lib, fn=fn, **kw) == expect


def _append(lib, fp8=False, ptrs=(P,) * 9, n=4, Hq=8, Hkv=2, d=128, rot=128, axes=1, qs=1536, ks=1536, vs=1536, bs=16,
            nblocks=10, scales=(0.5, 0.5)):
    q, k, v, pos, f, slots, qo, kc, vc = ptrs
    args = [q, k, v, pos, f, None, slots, n, Hq, Hkv, d, rot, axes, 4, qs, ks, vs, 0, bs, nblocks]
    if fp8:
        return lib.rope_axes_paged_append_fp8(*args, *[ctypes.c_float(s) for s in scales], qo, kc, vc, None)
    return lib.rope_axes_paged_append(*args, qo, kc, vc, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,expect", [
    *[(dict(ptrs=_p(i, None, 9)), INVALID) for i in range(9)],
    (dict(Hkv=0), INVALID),
    (dict(nblocks=0), INVALID),
    (dict(bs=0), INVALID),
    (dict(vs=128), INVALID),
    (dict(bs=8), UNSUPPORTED),
    (dict(nblocks=1 << 27), UNSUPPORTED),
    (dict(d=32, rot=32), UNSUPPORTED),
    (dict(vs=1540), UNSUPPORTED),
    (dict(ptrs=_p(7, P + 8, 9)), UNSUPPORTED),
    (dict(n=0), OK),
])
def test_append_refusals(lib, fp8, kw, expect):
    assert _append(lib, fp8=fp8, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(d=64, rot=64), UNSUPPORTED),
    (dict(scales=(0.0, 1.0)), INVALID),
    (dict(scales=(1.0, float("inf"))), INVALID),
    (dict(scales=(float("nan"), 1.0)), INVALID),
])
def test_append_fp8_refusals(lib, kw, expect):
    assert _append(lib, fp8=True, **kw) == expect


def _chunk(lib, checked=False, ptrs=(P,) * 8, B=2, Hq=8, Hkv=2, d=128, bs=16, maxb=8, nblocks=50, max_q=32, total_q=40,
           scale=0.088, ks=0.5, vs=0.5, splits=0):
    q, kc, vc, bt, sl, cq, o, lse = ptrs
    f = ctypes.c_float
    if checked:
        return lib.paged_attn_prefill_fp8_checked(q, kc, vc, bt, sl, cq, B, Hq, Hkv, d, bs, maxb, nblocks, max_q,
                                                  total_q, 1, f(scale), f(ks), f(vs), splits, o, lse, None)
    return lib.paged_attn_prefill_fp8(q, kc, vc, bt, sl, cq, B, Hq, Hkv, d, bs, maxb, max_q, total_q, 1, f(scale), f(ks),
                                      f(vs), splits, o, lse, None)


@pytest.mark.parametrize("checked", [False, True])
@pytest.mark.parametrize("kw,expect", [
    *[(dict(ptrs=_p(i, None, 8)), INVALID) for i in range(7)],
    (dict(scale=0.0), INVALID),
    (dict(ks=float("nan")), INVALID),
    (dict(vs=-1.0), INVALID),
    (dict(Hq=9), INVALID),
    (dict(maxb=0), INVALID),
    (dict(total_q=-1), INVALID),
    (dict(d=64), UNSUPPORTED),
    (dict(bs=32), UNSUPPORTED),
    (dict(maxb=1 << 27), UNSUPPORTED),
    (dict(Hq=129, Hkv=1), UNSUPPORTED),
    (dict(ptrs=_p(1, P + 8, 8)), UNSUPPORTED),
    (dict(ptrs=_p(7, P + 2, 8)), UNSUPPORTED),
    (dict(B=0), OK),
    (dict(total_q=0), OK),
    (dict(max_q=0), OK),
])
def test_prefill_fp8_refusals(lib, checked, kw, expect):
    assert _chunk(lib, checked=checked, **kw) == expect


def test_prefill_fp8_checked_pool(lib):
    assert _chunk(lib, checked=True, nblocks=0) == INVALID
    assert _chunk(lib, checked=True, nblocks=1 << 27) == UNSUPPORTED


def test_no_cpu_fallback(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc in (_plan(lib), _rope(lib), _append(lib), _append(lib, fp8=True), _chunk(lib), _chunk(lib, checked=True)):
        assert rc < 0


def test_axis_map():
    import flashattention_attention_attn_b200 as fa
    assert fa.rope_axis_map([2, 3, 1]) == bytes([0, 0, 1, 1, 1, 2])
    assert fa.rope_axis_map([3, 1, 2], interleaved=True) == bytes([0, 1, 2, 0, 2, 0])
    assert fa.rope_axis_map([4]) == bytes(4)
    with pytest.raises(ValueError):
        fa.rope_axis_map([-1, 2])
    with pytest.raises(ValueError):  # 64 pairs need 64 axes
        fa.rope_axes_fwd(None, None, None, None, bytes(10), 0, 8, 2, 128, 128, 1, 0, 1024, 256, False, None, None, 1024,
                         256, stream=0)


# ------------------------------------------------------------------ oracle pins
def test_oracle_plan_by_hand():
    table = [[7, 3, -1, -1], [-1, -1, -1, -1], [5, 9, -1, -1]]
    r = ps.plan_step([17, 0, 32], [2, 33, 1], [40, 41, 42, 43, 44], [0, 100, -1], table, 40)
    assert r["block_table"].tolist() == [[7, 3, -1, -1], [40, 41, 42, -1], [5, 9, 43, -1]]
    assert r["seq_lens"].tolist() == [19, 33, 33] and r["cu_seqlens_q"].tolist() == [0, 2, 35, 36]
    assert r["slot_map"].tolist() == [49, 50] + list(range(640, 673)) + [688] + [-1] * 4
    assert r["positions"].tolist() == [17, 18] + list(range(100, 133)) + [31] + [0] * 4
    assert r["blocks_taken"].tolist() == [4] and not r["flags"]


def test_oracle_plan_flags():
    r = ps.plan_step([0, 0], [20, 20], [1, 2, 3], None, [[-1] * 2] * 2, 64)
    assert r["flags"] == {"noblock"} and r["block_table"].tolist() == [[1, 2], [3, -1]]
    assert r["slot_map"][36:40].tolist() == [-1] * 4 and r["blocks_taken"].tolist() == [4]
    r = ps.plan_step([30], [5], [], None, [[4, 6]], 8)  # three tokens past the row
    assert r["flags"] == {"seqlen"} and r["seq_lens"].tolist() == [32]
    assert r["slot_map"].tolist() == [110, 111, -1, -1, -1, -1, -1, -1]
    r = ps.plan_step([5], [1], [], None, [[-1]], 1)
    assert r["flags"] == {"badblock"} and r["slot_map"].tolist() == [-1]


def test_oracle_rope_is_a_rotation():
    g = np.random.default_rng(0)
    x = g.standard_normal((5, 3, 64))
    pos = g.integers(0, 1000, (2, 5))
    f = 10000.0 ** (-np.arange(16) / 16)
    axis = [0] * 6 + [1] * 10
    for adjacent in (False, True):
        y = ps.rope_axes(x, pos, f, axis, adjacent)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose(ps.rope_axes(y, pos, f, axis, adjacent, sign=-1.0), x, atol=1e-12)
        # a dot product depends on the difference of the positions alone
        a = (ps.rope_axes(x, pos + 7, f, axis, adjacent)[:, 0] * ps.rope_axes(x, pos + 4, f, axis, adjacent)[:, 1]).sum(-1)
        b = (ps.rope_axes(x, 0 * pos + 3, f, axis, adjacent)[:, 0] * x[:, 1]).sum(-1)
        assert np.allclose(a, b)
        one = ps.rope_axes(np.eye(64)[None, :1], np.array([[1], [2]]), f, axis, adjacent)[0, 0]
        assert np.isclose(one[0], np.cos(1.0)) and np.isclose(one[1 if adjacent else 16], np.sin(1.0))


def test_oracle_e4m3_against_torch():
    v = ps.e4m3_values()
    assert np.array_equal(v, orc.decode_e4m3(np.arange(127, dtype=np.uint8)))
    x = np.concatenate([np.random.default_rng(1).standard_normal(5000) * s for s in (1e-3, 0.1, 1, 60)] +
                       [v, -v, (v[1:] + v[:-1]) / 2])
    t = torch.from_numpy(x).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ps.nearest_e4m3(x.astype(np.float32)), t)


@pytest.mark.parametrize("scale,ks", [(1e30, 1e30), (3e38, 1.0)])
def test_prefill_fp8_refuses_a_product_of_scales_past_fp32(lib, scale, ks):
    assert _chunk(lib, scale=scale, ks=ks) == INVALID


def test_ops_refuse_sizes_that_do_not_fit():
    """What a call would read past: refused before anything is launched."""
    import flashattention_attention_attn_b200.torch_ops  # noqa: F401
    ops = torch.ops.fa_b200
    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    B, n = 3, 10
    table, lens, free, f = torch.zeros(B, 4, **i32), torch.zeros(B, **i32), torch.zeros(9, **i32), torch.ones(64)
    q, k, pos, slots = torch.zeros(n, 4, 128, **bf), torch.zeros(n, 2, 128, **bf), torch.zeros(2, n, **i32), torch.zeros(n, **i32)
    kc, k8 = torch.zeros(9, 16, 2, 128, **bf), torch.zeros(9, 16, 2, 128, dtype=torch.uint8)
    cu = torch.zeros(B + 1, **i32)

    def refused(name, op, *args):
        with pytest.raises(ValueError, match=name):
            op(*args)

    refused("new_lens", ops.paged_cache_plan, table, lens, lens[:2], free, None, n)
    refused("cached_lens", ops.paged_cache_plan, table, cu, lens, free, None, n)
    refused("pos_offsets", ops.paged_cache_plan, table, lens, lens, free, cu, n)
    refused("block_table", ops.paged_cache_plan, lens, lens, lens, free, None, n)
    refused("k is", ops.rope_axes, q, k[:9], pos, f, [], False)
    refused("k is", ops.rope_axes, q, torch.zeros(n, 2, 64, **bf), pos, f, [], False)
    refused("positions", ops.rope_axes, q, k, pos[:, :9], f, [], False)
    refused("positions", ops.rope_axes, q, k, pos[0], f, [], False)
    for op, c, scales in ((ops.rope_axes_paged_append, kc, ()), (ops.rope_axes_paged_append_fp8, k8, (1.0, 1.0))):
        refused("slot_map", op, q, k, k, pos, f, [], slots[:9], False, c, c.clone(), *scales)
        refused("v is", op, q, k, q, pos, f, [], slots, False, c, c.clone(), *scales)
        refused("k is", op, q, q, k, pos, f, [], slots, False, c, c.clone(), *scales)
        refused("v_cache", op, q, k, k, pos, f, [], slots, False, c, c[:8].clone(), *scales)
    args = (True, 0.1, 1.0, 1.0, 0)
    refused("v_cache", ops.paged_attn_prefill_fp8, q, k8, k8[:5], table, lens, cu, 8, *args)
    refused("k_cache", ops.paged_attn_prefill_fp8, q[..., :64], k8, k8, table, lens, cu, 8, *args)
    refused("block_table", ops.paged_attn_prefill_fp8, q, k8, k8, table[:2], lens, cu, 8, *args)
    refused("seq_lens", ops.paged_attn_prefill_fp8, q, k8, k8, table, cu, cu, 8, *args)
