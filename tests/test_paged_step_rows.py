"""The torch ops of the serving step on rows that lie off a 16-byte boundary."""

import pytest
import torch

BF16 = torch.bfloat16


def off_boundary(x):
    """The values of x, packed, in a buffer that is one element further on than the allocation."""
    flat = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)
    flat[1:] = x.reshape(-1)
    return flat[1:].view(x.shape)


def test_rows_off_the_boundary_are_copied():
    from flashattention_attention_attn_b200 import torch_ops
    x = torch.arange(3 * 2 * 64).to(BF16).view(3, 2, 64)
    y = off_boundary(x)
    assert y.is_contiguous() and y.data_ptr() % 16 != 0
    for f in (torch_ops._rows, torch_ops._packed):
        assert f(y).data_ptr() % 16 == 0 and torch.equal(f(y), x)
        assert f(x).data_ptr() == x.data_ptr()  # and only those
    gap = torch.cat([x, x], 1)[:, :2]  # rows apart, on the boundary: as they are for the rotary calls
    assert torch_ops._rows(gap).data_ptr() == gap.data_ptr() and torch_ops._packed(gap).is_contiguous()
    shifted = torch.cat([x, x], 2)[..., 4:68]
    assert torch_ops._rows(shifted).data_ptr() % 16 == 0 and torch.equal(torch_ops._rows(shifted), shifted)


@pytest.mark.gpu
def test_ops_take_rows_off_the_boundary():
    import flashattention_attention_attn_b200.torch_ops  # noqa: F401
    ops = torch.ops.fa_b200
    g = torch.Generator().manual_seed(4)
    n, H, d, pool = 9, 4, 128, 3
    q, k, v, dy = (torch.randn(n, H, d, generator=g).to(BF16).cuda() for _ in range(4))
    f, pos = torch.rand(d // 2, generator=g).cuda(), torch.arange(n, dtype=torch.int32, device="cuda")
    args = (pos[None], f, [], False)
    want = ops.rope_axes(q, k, *args)
    got = ops.rope_axes(off_boundary(q), off_boundary(k), *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    grads = []
    for y in (dy, off_boundary(dy)):
        a, b = q.clone().requires_grad_(), k.clone().requires_grad_()
        grads.append(torch.autograd.grad(ops.rope_axes(a, b, *args), (a, b), (y, y)))
    assert all(torch.equal(x, y) for x, y in zip(*grads))
    outs = []
    for move in (lambda x: x, off_boundary):
        kc, vc = (torch.zeros(pool, 16, H, d, dtype=torch.uint8, device="cuda") for _ in range(2))
        qr = ops.rope_axes_paged_append_fp8(move(q), move(k), move(v), pos[None], f, [], pos, False, kc, vc, 0.02, 0.02)
        table = torch.arange(pool, dtype=torch.int32, device="cuda")[None]
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        outs.append((qr, kc, vc, *ops.paged_attn_prefill_fp8(move(qr), kc, vc, table, lens, cu, n, True, 0.09, 0.02, 0.02,
                                                             0)))
    assert all(torch.equal(x, y) for x, y in zip(*outs))
