"""The operators together, as a program uses them: a layer for serving in 8-bit
integers, and a training step of one, put together from parts."""

from __future__ import annotations

import pytest
import torch

import sort_reference as sref
import swiglu_reference as gref
from gpu_helpers import log
from mixture_experts_expert_mm_amd import moe
from sort_reference import F64, HALF, U32

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(y, want, err, what):
    over = (y.detach().cpu().to(F64) - want).abs() - err
    assert bool((over <= 0).all()), (what, float(over.max()), float(want.abs().max()))


def weights(E, H, I, seed):
    """Formula-layout weights as int8 codes with a scale per output channel."""
    g = gen(seed)
    w1, s1 = gref.codes(torch.randn(E, 2 * I, H, generator=g) * H ** -0.5)
    w2, s2 = gref.codes(torch.randn(E, H, I, generator=g) * I ** -0.5)
    return w1, s1, w2, s2


def product(x, w, ws, off, cnt):
    """Grouped int8 product in 64 bits from floating rows, and its error."""
    q, s = gref.codes(x)
    y = torch.zeros(x.shape[0], w.shape[1], dtype=F64)
    for i in range(w.shape[0]):
        lo, hi = int(off[i]), int(off[i] + cnt[i])
        y[lo:hi] = (q[lo:hi].to(F64) @ w[i].to(F64).t()) * ws[i].to(F64) * s[lo:hi].to(F64)[:, None]
    return y, y.abs() * (3 * U32 + HALF[BF16]) * 1.01


@pytest.mark.parametrize("T,H,I,E,K", [(1, 512, 128, 8, 2), (37, 256, 256, 6, 3), (700, 512, 384, 16, 4), (3000, 256, 128, 8, 4)])
def test_serving(T, H, I, E, K):
    """route, sort, product, activation, product, back: each step against its formula on the step's own inputs; the
    whole against the library's int8 layer on the same weights."""
    log(f"[parts serving] T={T} H={H} I={I} E={E} K={K}")
    g = gen(T)
    x = torch.randn(T, H, generator=g).to(BF16)
    w1, s1, w2, s2 = weights(E, H, I, 5)
    wr = (torch.randn(E, H, generator=g) * H ** -0.5).to(BF16)
    active = (torch.rand(T, generator=g) > 0.1).to(torch.int8)
    active[0] = 1
    w1d, s1d, w2d, s2d = (t.cuda() for t in (w1, s1, w2, s2))

    def step(x, active):
        ids, gates = moe.route(x, wr.cuda(), topk=K, active=active)
        rows, o = moe.sort_tokens(x, ids, E, active=active)
        h = moe.int8_linear(rows, w1d, s1d, o.offsets, o.counts)
        a = moe.swiglu(h)
        r = moe.int8_linear(a, w2d, s2d, o.offsets, o.counts)
        return ids, gates, rows, o, h, a, r, moe.combine_tokens(r, o, gates)

    ids, gates, rows, o, h, a, r, y = step(x.cuda(), active.cuda())
    order = sref.order(ids.cpu(), E, active)
    n = int(order[1][-1])
    assert torch.equal(rows.cpu(), sref.rows_of(x, order[3], K))
    want, err = product(rows.cpu()[:n], w1, s1, order[1], order[0])
    within(h[:n], want, err, "Linear1")
    within(a[:n], *gref.forward(h.cpu()[:n]), "activation")
    want, err = product(a.cpu()[:n], w2, s2, order[1], order[0])
    within(r[:n], want, err, "Linear2")
    within(y, *sref.combine(r.cpu(), order[2], gates.cpu()), "combine")
    assert bool((y[active.cuda() == 0] == 0).all())
    # codes sorted after quantising are the same product
    q, s = moe.int8_quantize(x.cuda())
    h2 = moe.int8_matmul(moe.sort_rows(q, o), moe.sort_rows(s[:, None], o).view(-1), w1d, s1d, o.offsets, o.counts)
    assert torch.equal(h2[:n], h[:n])
    layer = moe.ExpertLayer(T, H, I, E, K, "int8")
    layer.load_weights(w1.transpose(1, 2).contiguous(), w2.transpose(1, 2).contiguous(), s1, s2)
    # the parts on the layer's own weights: gate and up columns alternate, and so do their scales
    turn = layer.plan.gate_up_group
    s1_turned = layer.s1.view(E, 2, I // turn, turn).transpose(1, 2).reshape(E, 2 * I).contiguous()
    a2 = moe.swiglu(moe.int8_linear(rows, layer.w1, s1_turned, o.offsets, o.counts), gate_up_group=turn)
    assert torch.equal(a2[:n], a[:n])
    assert torch.equal(moe.combine_tokens(moe.int8_linear(a2, layer.w2, layer.s2, o.offsets, o.counts), o, gates), y)
    whole, counts = layer.forward(x.cuda(), ids, gates, active=active.cuda())
    assert torch.equal(counts, o.counts)
    # The layer quantises its float32 SwiGLU(h); the parts round h and a to bf16 first.  With |silu'| <= 1.1 and
    # |silu(g)| <= |g|, half a step of bf16 in g and u moves a by at most (1.1 + 1) 2^-8 |g u|, its own rounding by
    # 2^-8 |a|, and each side's code is within half a scale of its value; scales differ by less than a tenth.  These
    # move a route's row by at most their sum over |W2|; both sides' routes and sums are rounded to bf16.
    hn, an = h.cpu()[:n].to(F64).abs(), a.cpu()[:n].to(F64).abs()
    half = HALF[BF16]
    delta = 2.1 * 1.02 * half * hn[:, :I] * hn[:, I:] + half * an + 1.1 * gref.codes(a.cpu()[:n])[1].to(F64)[:, None]
    moved = torch.zeros(T * K, H, dtype=F64)
    for e in range(E):
        lo, hi = int(order[1][e]), int(order[1][e + 1])
        moved[lo:hi] = delta[lo:hi] @ (w2[e].to(F64).abs() * s2[e].to(F64)[:, None]).t()
    moved[:n] += 2 * half * (r.cpu()[:n].to(F64).abs() + moved[:n])
    bound, _ = sref.combine(moved, order[2], gates.cpu(), dtype=BF16)
    within(whole, y.cpu().to(F64), bound + 2 * half * (y.cpu().to(F64).abs() + bound), "layer")


def test_serving_in_a_graph():
    """The whole step captured once and replayed on other tokens."""
    T, H, I, E, K = 300, 256, 128, 8, 2
    w1, s1, w2, s2 = (t.cuda() for t in weights(E, H, I, 5))
    wr = (torch.randn(E, H, generator=gen(1)) * H ** -0.5).to(BF16).cuda()

    def step(x):
        ids, gates = moe.route(x, wr, topk=K)
        rows, o = moe.sort_tokens(x, ids, E)
        a = moe.swiglu(moe.int8_linear(rows, w1, s1, o.offsets, o.counts))
        return moe.combine_tokens(moe.int8_linear(a, w2, s2, o.offsets, o.counts), o, gates)

    xs = [torch.randn(T, H, generator=gen(i)).to(BF16).cuda() for i in range(3)]
    want = [step(x) for x in xs]
    buf = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(buf)
    for i in (1, 2, 0, 1):
        buf.copy_(xs[i])
        graph.replay()
        again = step(xs[2 - i])
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]) and torch.equal(again, want[2 - i])


@pytest.mark.parametrize("T,H,I,E,K,clamp", [(5, 32, 24, 3, 2, None), (60, 48, 130, 4, 3, 1.0), (400, 64, 128, 8, 2, None)])
def test_training_step(T, H, I, E, K, clamp):
    """Gradients of x, the gates and the weights through the whole layer in float32, against 64-bit formulas with the
    activation's gradient at its kept values."""
    log(f"[parts training] T={T} H={H} I={I} E={E} K={K}")
    g = gen(T)
    x = torch.randn(T, H, generator=g)
    w1 = torch.randn(E, 2 * I, H, generator=g) * H ** -0.5
    w2 = torch.randn(E, H, I, generator=g) * I ** -0.5
    gates = torch.softmax(torch.randn(T, K, generator=g), 1)
    ids = torch.randn(T, E, generator=g).argsort(1)[:, :K].to(torch.int32)
    ids[torch.rand(T, K, generator=g) < 0.1] = -1
    dy = torch.randn(T, H, generator=g)
    leaves = [t.cuda().requires_grad_() for t in (x, w1, w2, gates)]
    xd, w1d, w2d, gd = leaves
    rows, o = moe.sort_tokens(xd, ids.cuda(), E)
    off = o.offsets.tolist()
    per_expert = lambda t, w: torch.cat([t[off[e]:off[e + 1]] @ w[e].t() for e in range(E)] + [t.new_zeros(T * K - off[E], w.shape[1])])
    h = per_expert(rows, w1d)
    r = per_expert(moe.swiglu(h, activation_clamp=clamp), w2d)
    y = moe.combine_tokens(r, o, gd)
    grads = torch.autograd.grad(y, leaves, dy.cuda())

    def chain(x, w1, w2, gates, dy, h0, absolute):
        """All gradients in 64 bits; with `absolute`, of the magnitudes: bounds every partial sum."""
        f = torch.abs if absolute else (lambda t: t)
        x, w1, w2, gates, dy = (f(t.to(F64)) for t in (x, w1, w2, gates, dy))
        counts, offsets, row, route = sref.order(ids, E)
        n = int(offsets[-1])
        tok, rt = route[:n].long() // K, route[:n].long()
        expert = torch.repeat_interleave(torch.arange(E), counts.long())
        a = f(gref.forward(h0[:n], clamp)[0])
        d = dy[tok]
        gate = gates.reshape(-1)[rt][:, None]
        r = torch.einsum("nhi,ni->nh", w2[expert], a)
        dgates = torch.zeros(T * K, dtype=F64)
        dgates[rt] = (d * r).sum(1)
        dr = d * gate
        dw2 = torch.zeros_like(w2).index_add_(0, expert, dr[:, :, None] * a[:, None, :])
        da = torch.einsum("nhi,nh->ni", w2[expert], dr)
        q, s = gref.keep(h0[:n])
        if absolute:                     # |d a / d g| <= 1.1 |u|, |d a / d u| <= |g| at the kept values
            v = gref.kept(q, s).to(F64).abs()
            dh = torch.cat([da * 1.1 * v[:, I:], da * v[:, :I]], 1)
        else:
            dh = exact_backward(da, q, s)
        dw1 = torch.zeros_like(w1).index_add_(0, expert, dh[:, :, None] * x[tok][:, None, :])
        dx = torch.zeros_like(x).index_add_(0, tok, torch.einsum("noh,no->nh", w1[expert], dh))
        return dx, dw1, dw2, dgates.view(T, K)

    def exact_backward(da, q, s):
        lim = gref.clamp_of(clamp)
        v = gref.kept(q, s).to(F64)
        g0, u0 = v[:, :I], v[:, I:]
        g, u = g0.clamp(-lim, lim), u0.clamp(-lim, lim)
        sig = torch.sigmoid(g)
        return torch.cat([da * u * sig * (1 + g * (1 - sig)) * (g0.abs() <= lim), da * g * sig * (u0.abs() <= lim)], 1)

    h0 = h.detach().cpu()
    want = chain(x, w1, w2, gates, dy, h0, False)
    mag = chain(x, w1, w2, gates, dy, h0, True)
    # sums of at most 2 I + H + I + T K terms one after the other along a path, a sigmoid and a few products, each step
    # within one unit (2 U32, truncation allowed) of partial sums that the magnitudes' chain bounds
    steps = 2 * I + H + I + T * K + 40
    for got, w, m, name in zip(grads, want, mag, ("x", "w1", "w2", "gates")):
        within(got, w, steps * 2 * U32 * m, name)
