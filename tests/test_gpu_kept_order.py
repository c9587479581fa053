"""What the differentiable functions keep for their backward pass, on the GPU:
gradients go by the forward call's order, also where the program has used its
objects again, moved what is kept to the host, or computes the forward pass anew."""

from __future__ import annotations

import pytest
import torch
from torch.utils.checkpoint import checkpoint

import sort_reference as ref
from mixture_experts_expert_mm_amd import moe

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(y, want, err):
    over = (y.detach().cpu().to(F64) - want).abs() - err
    assert bool((over <= 0).all()), (float(over.max()), float(want.abs().max()))


def batch(T, H, E, K, seed):
    g = gen(seed)
    ids = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32)
    return (ids, torch.randn(T, H, generator=g).to(BF16), torch.rand(T, K, generator=g), torch.randn(T * K, H, generator=g).to(BF16),
            torch.randn(T, H, generator=g).to(BF16))


@pytest.mark.parametrize("T", [40, 1500])                    # the order in one launch, and in several
def test_an_order_used_again(T):
    """The next, smaller micro-batch's order in the same object, and its statistics written over."""
    H, E, K = 48, 6, 3
    ids, x, w, rows, dy = batch(T, H, E, K, T)
    want = ref.order(ids, E)
    xr, rr, wr, pr = (t.cuda().requires_grad_() for t in (x, rows, w, rows))
    a, o = moe.sort_tokens(xr, ids.cuda(), E)
    b, y, z = moe.sort_rows(xr, o), moe.combine_tokens(rr, o, wr), moe.combine_tokens(pr, o)
    _, other = moe.sort_tokens(x[:T // 2].cuda(), batch(T // 2, H, E, K, 1)[0].cuda(), E)
    o.counts, o.offsets, o.row_of_route, o.route_of_row = other.counts, other.offsets, other.row_of_route, other.route_of_row
    torch.autograd.backward((y, z), (dy.cuda(), dy.cuda()))
    drows, derr, dw, werr = ref.combine_backward(dy, rows, want[2], w)
    within(rr.grad, drows, derr)
    within(wr.grad, dw, werr)
    assert torch.equal(pr.grad.cpu(), ref.rows_of(dy, want[3], K))
    dx, err = ref.combine(rows, want[2])
    for t in (a, b):
        within(torch.autograd.grad(t, xr, rows.cuda())[0], dx, err)


def test_kept_on_the_host_and_computed_anew():
    T, H, E, K = 300, 64, 5, 2
    ids, x, w, _, dy = batch(T, H, E, K, 3)
    ids, dy = ids.cuda(), dy[:, :H // 2].contiguous().cuda()

    def step(x, w):
        rows, o = moe.sort_tokens(x, ids, E)
        return moe.combine_tokens(moe.swiglu(rows), o, w)

    leaves = [t.cuda().requires_grad_() for t in (x, w)]
    want = torch.autograd.grad(step(*leaves), leaves, dy)
    with torch.autograd.graph.save_on_cpu():
        y = step(*leaves)
    for got in (torch.autograd.grad(y, leaves, dy),
                torch.autograd.grad(checkpoint(step, *leaves, use_reentrant=False), leaves, dy)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_an_order_made_in_inference_mode():
    T, H, E, K = 70, 32, 5, 2
    ids, x, w, rows, dy = batch(T, H, E, K, 4)
    with torch.inference_mode():
        _, o = moe.sort_tokens(x.cuda(), ids.cuda(), E)
    rr, wr = rows.cuda().requires_grad_(), w.cuda().requires_grad_()
    moe.combine_tokens(rr, o, wr).backward(dy.cuda())
    drows, derr, dw, werr = ref.combine_backward(dy, rows, ref.order(ids, E)[2], w)
    within(rr.grad, drows, derr)
    within(wr.grad, dw, werr)
