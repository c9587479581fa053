"""Tokens sorted by expert and back, and their gradients, on the GPU against
plain implementations, at the sizes and masks where they can go wrong."""

from __future__ import annotations

import pytest
import torch

import sort_reference as ref
from gpu_helpers import log
from mixture_experts_expert_mm_amd import moe

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def routes(T, E, K, seed, kind="spread"):
    g = gen(seed)
    if kind == "one":                     # every route to one expert
        return torch.full((T, K), E - 1, dtype=torch.int32), None
    if kind == "none":                    # nothing is kept
        return torch.randint(-3, 0, (T, K), generator=g, dtype=torch.int32), None
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)     # a token may name an expert twice
    if kind == "masked":
        u = torch.rand(T, K, generator=g)
        ids[u < 0.1] = -1
        ids[(u >= 0.1) & (u < 0.15)] = E
        ids[(u >= 0.15) & (u < 0.2)] = 2 ** 31 - 1
        ids[(u >= 0.2) & (u < 0.25)] = -2 ** 31
        return ids, (torch.rand(T, generator=g) > 0.2).to(torch.int8) * 3
    return ids, None


def cuda(t):
    return None if t is None else t.cuda()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def same(order, want):
    for got, w in zip((order.counts, order.offsets, order.row_of_route, order.route_of_row), want):
        assert torch.equal(got.cpu(), w)


def within(y, want, err):
    over = (y.detach().cpu().to(F64) - want).abs() - err
    assert bool((over <= 0).all()), (float(over.max()), float(want.abs().max()))


# around the limit of the single launch (4096 routes for each eight slots), of a chunk (1024) and of a turn; E around the waves' and
# workgroups' sizes
SHAPES = [(1, 8, 1, 1), (1, 7168, 32, 8), (3, 1, 5, 5), (17, 33, 8, 4), (64, 520, 1024, 64), (129, 6, 257, 3),
          (1024, 16, 64, 8), (1025, 16, 64, 8), (8193, 4, 255, 1), (2731, 3, 1000, 3), (20011, 2, 16, 5), (700, 1, 1024, 64),
          (5000, 256, 256, 8), (40000, 8, 3, 2), (512, 520, 40, 8), (513, 520, 40, 8), (227, 64, 99, 9), (228, 64, 99, 9)]


@pytest.mark.parametrize("T,H,E,K", SHAPES)
@pytest.mark.parametrize("kind", ["spread", "masked"])
def test_sort(T, H, E, K, kind):
    log(f"[sort] T={T} H={H} E={E} K={K} {kind}")
    ids, active = routes(T, E, K, T + E, kind)
    want = ref.order(ids, E, active)
    x = torch.randn(T, H, generator=gen(T)).to(BF16)
    rows, order = moe.sort_tokens(x.cuda(), ids.cuda(), E, active=cuda(active))
    same(order, want)
    assert torch.equal(bits(rows), bits(ref.rows_of(x, want[3], K)))
    # the same order for another tensor
    s = torch.randn(T, 1, generator=gen(T + 1))
    assert torch.equal(moe.sort_rows(s.cuda(), order).cpu(), ref.rows_of(s, want[3], K))


@pytest.mark.parametrize("kind", ["one", "none"])
@pytest.mark.parametrize("T", [5, 9000])
def test_sort_one_expert_and_none(T, kind):
    ids, _ = routes(T, 6, 3, T, kind)
    x = torch.randn(T, 40, generator=gen(T)).to(F16)
    want = ref.order(ids, 6)
    rows, order = moe.sort_tokens(x.cuda(), ids.cuda(), 6)
    same(order, want)
    assert torch.equal(bits(rows), bits(ref.rows_of(x, want[3], 3)))
    y = moe.combine_tokens(rows, order, torch.full((T, 3), float("nan"), device="cuda") if kind == "none" else None)
    if kind == "none":
        assert bool((y == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32, torch.int8, torch.uint8, E4M3])
@pytest.mark.parametrize("T,H", [(7, 1), (33, 18), (2100, 20), (2100, 7), (40, 4096), (2100, 2048)])
def test_types_and_widths(dtype, T, H):
    ids, active = routes(T, 9, 4, H, "masked")
    raw = torch.randint(0, 120, (T, H * dtype.itemsize), generator=gen(3), dtype=torch.uint8)   # no NaN of any type
    x = raw.view(dtype).view(T, H)
    rows, order = moe.sort_tokens(x.cuda(), ids.cuda(), 9, active=cuda(active))
    want = ref.order(ids, 9, active)
    same(order, want)
    assert torch.equal(bits(rows), bits(ref.rows_of(raw, want[3], 4).view(dtype)))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,H,E,K,kind", [(1, 7168, 32, 8, "spread"), (3, 1, 5, 5, "masked"), (65, 33, 8, 4, "masked"), (200, 520, 32, 17, "masked"),
                                          (130, 2050, 16, 8, "spread"), (2100, 12, 9, 64, "masked"), (300, 4096, 16, 4, "masked"),
                                          (40, 2046, 4, 9, "masked"), (7, 300, 3, 2, "none")])
def test_combine_and_gradients(dtype, T, H, E, K, kind):
    log(f"[combine] T={T} H={H} E={E} K={K} {kind} {dtype}")
    ids, active = routes(T, E, K, T + H, kind)
    g = gen(H)
    rows = torch.randn(T * K, H, generator=g).to(dtype)
    w = torch.rand(T, K, generator=g) - 0.2
    dy = torch.randn(T, H, generator=g).to(dtype)
    want = ref.order(ids, E, active)
    order = moe.TokenOrder(*(t.cuda() for t in want))
    kept = int(want[1][-1])
    dead = rows.clone()
    dead[kept:] = float("nan")           # rows that no route fills are never read
    wd = w.clone()
    wd[want[2] < 0] = float("inf")       # nor are the weights of skipped routes
    for weights in (None, wd):
        y, err = ref.combine(rows, want[2], None if weights is None else w)
        within(moe.combine_tokens(dead.cuda(), order, cuda(weights)), y, err)
    drows, derr, dw, werr = ref.combine_backward(dy, rows, want[2], w)
    got = moe.combine_backward(dy.cuda(), dead.cuda(), order, wd.cuda())
    within(got[0], drows, derr)
    within(got[1], dw, werr)
    # autograd gives the same, with each of the inputs alone too
    for of in ("rows", "weights", "both"):
        r, q = dead.cuda().requires_grad_(of != "weights"), wd.cuda().requires_grad_(of != "rows")
        moe.combine_tokens(r, order, q).backward(dy.cuda())
        if of != "weights":
            assert torch.equal(bits(r.grad), bits(got[0]))
        if of != "rows":
            assert torch.equal(q.grad, got[1])
    r = dead.cuda().requires_grad_()
    moe.combine_tokens(r, order).backward(dy.cuda())
    assert torch.equal(bits(r.grad), bits(ref.rows_of(dy, want[3], K)))
    # the sort's gradient
    x = torch.randn(T, H, generator=g).to(dtype).cuda().requires_grad_()
    sorted_rows, o = moe.sort_tokens(x, ids.cuda(), E, active=cuda(active))
    same(o, want)
    sorted_rows.backward(dead.cuda())
    y, err = ref.combine(rows, want[2])
    within(x.grad, y, err)


def test_gradients_against_differences():
    """sum of squares of a sorted, weighted and combined batch: its slope along random directions."""
    g = gen(5)
    T, H, E, K = 9, 12, 4, 3
    ids, active = routes(T, E, K, 1, "masked")
    x, w = torch.randn(T, H, generator=g).cuda(), torch.rand(T, K, generator=g).cuda()

    def f(x, w):
        rows, order = moe.sort_tokens(x, ids.cuda(), E, active=active.cuda())
        return (moe.combine_tokens(rows * 1.5, order, w).double() ** 2).sum()

    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    gx, gw = torch.autograd.grad(f(xr, wr), (xr, wr))
    for seed in range(4):
        dx, dw = torch.randn(T, H, generator=gen(seed)).cuda(), torch.randn(T, K, generator=gen(seed + 9)).cuda()
        h = 2.0 ** -6
        slope = (f(x + h * dx, w + h * dw) - f(x - h * dx, w - h * dw)) / (2 * h)
        want = (gx * dx).double().sum() + (gw * dw).double().sum()
        # f is a polynomial of degree 4 in h: the odd rest is h^2 times the slope's third-order term, f(dx, dw)'s size;
        # float32 rounding of f adds 2^-24 of f / h
        rest = h * h * 4 * (f(x.abs() + dx.abs(), w + dw.abs()))
        assert abs(float(slope - want)) <= float(rest) + 2.0 ** -24 * float(f(x, w)) / h * 16


def test_shared_and_expanded_gradients():
    """Gradients that reach the operators expanded, strided or at an odd address, and rows that two calls share."""
    T, H, E, K = 50, 24, 4, 3
    ids, active = routes(T, E, K, 2, "masked")
    g = gen(8)
    want = ref.order(ids, E, active)
    order = moe.TokenOrder(*(t.cuda() for t in want))
    base, w = torch.randn(T * K, H, generator=g), torch.rand(T, K, generator=g)
    for dtype in (BF16, F32):
        rows = base.to(dtype)
        r, q = rows.cuda().requires_grad_(), w.cuda().requires_grad_()
        moe.combine_tokens(r, order, q).sum().backward()           # an expanded scalar
        drows, derr, dw, werr = ref.combine_backward(torch.ones(T, H, dtype=dtype), rows, want[2], w)
        within(r.grad, drows, derr)
        within(q.grad, dw, werr)
        buf = torch.randn(T * H + 1, generator=gen(1)).to(dtype).cuda()
        for dy in (buf[1:].view(T, H), buf[1:].view(H, T).t()):
            r = rows.cuda().requires_grad_()
            moe.combine_tokens(r, order, w.cuda()).backward(dy)
            within(r.grad, *ref.combine_backward(dy.cpu(), rows, want[2], w)[:2])
        x = base[:T].to(dtype).cuda().requires_grad_()
        a, b = moe.sort_tokens(x, ids.cuda(), E, active=active.cuda())[0], moe.sort_rows(x, order)
        (a.float().sum() + 2 * b.float().sum()).backward()
        kept = (want[2] >= 0).sum(1).to(F64)[:, None].expand(T, H)
        assert torch.equal(x.grad.cpu().to(F64), 3 * kept)         # small whole numbers


def test_empty_batch():
    x, ids = torch.zeros(0, 16, dtype=BF16, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    rows, order = moe.sort_tokens(x, ids, 5)
    assert rows.shape == (0, 16) and bool((order.counts == 0).all()) and bool((order.offsets == 0).all())
    assert order.row_of_route.shape == (0, 2) and order.route_of_row.shape == (0,)
    w = torch.zeros(0, 2, device="cuda", requires_grad=True)
    y = moe.combine_tokens(rows.requires_grad_(), order, w)
    assert y.shape == (0, 16)
    y.sum().backward()
    assert w.grad.shape == (0, 2) and moe.sort_rows(x, order).shape == (0, 16)


def test_streams_and_graphs():
    """Another stream, given or current; captured calls replay with other inputs, two graphs with eager work between."""
    T, H, E, K = 1500, 96, 32, 8                              # the path of several launches
    g = gen(4)
    ids = [routes(T, E, K, s, "masked")[0] for s in range(3)]
    xs = [torch.randn(T, H, generator=g).to(BF16) for _ in range(3)]
    w = torch.rand(T, K, generator=g).cuda()
    dy = torch.randn(T, H, generator=g).to(BF16).cuda()

    def step(x, i):
        rows, o = moe.sort_tokens(x, i, E)
        y = moe.combine_tokens(rows, o, w)
        return rows, o.counts, o.offsets, o.row_of_route, o.route_of_row, y, *moe.combine_backward(dy, rows, o, w)

    want = [step(x.cuda(), i.cuda()) for x, i in zip(xs, ids)]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x, i = xs[0].cuda(), ids[0].cuda()
    rows, o = moe.sort_tokens(x, i, E, stream=s)
    y = moe.combine_tokens(rows, o, w, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(rows, want[0][0]) and torch.equal(y, want[0][5])
    xb, ib = xs[0].cuda(), ids[0].cuda()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(xb, ib)
        graphs.append((graph, out))
    for turn in range(3):
        for graph, out in graphs:
            xb.copy_(xs[turn])
            ib.copy_(ids[turn])
            graph.replay()
            eager = step(xb, ib)                              # between the replays
            torch.cuda.synchronize()
            for a, b, c in zip(out, want[turn], eager):
                assert torch.equal(a, b) and torch.equal(c, b)


def test_capture_with_autograd_is_refused():
    ids, _ = routes(6, 3, 2, 1)
    x = torch.randn(6, 8, device="cuda", requires_grad=True)
    rows, order = moe.sort_tokens(x.detach(), ids.cuda(), 3)
    w = torch.rand(6, 2, device="cuda", requires_grad=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in (lambda: moe.sort_tokens(x, ids, 3), lambda: moe.sort_rows(x, order),
                     lambda: moe.combine_tokens(rows, order, w)):
            with pytest.raises((RuntimeError, ValueError), match="capture|topk_ids"):
                call()
        with torch.no_grad():
            y = moe.combine_tokens(rows, order, w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, moe.combine_tokens(rows, order, w).detach())


def test_backward_twice_and_orders_written_over():
    """A graph may be kept and gone through again, not differentiated twice; an order may not change in between."""
    ids, _ = routes(40, 5, 3, 7)
    x = torch.randn(40, 16, device="cuda", requires_grad=True)
    w = torch.rand(40, 3, device="cuda", requires_grad=True)
    rows, order = moe.sort_tokens(x, ids.cuda(), 5)
    y = moe.combine_tokens(rows, order, w)
    dy = torch.randn_like(y)
    one = torch.autograd.grad(y, (x, w), dy, retain_graph=True)
    two = torch.autograd.grad(y, (x, w), dy, retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    three = torch.autograd.grad(y, (x, w), dy, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(one, three))
    with pytest.raises(RuntimeError, match="once_differentiable|does not require grad"):
        torch.autograd.grad(three[1].sum(), x)
    for t in (order.row_of_route, order.offsets):
        rows, order = moe.sort_tokens(x, ids.cuda(), 5)
        y = moe.combine_tokens(rows, order, w)
        {True: order.row_of_route, False: order.offsets}[t.dim() == 2].zero_()
        with pytest.raises(RuntimeError, match="modified in place"):
            torch.autograd.grad(y, (x, w), dy)
