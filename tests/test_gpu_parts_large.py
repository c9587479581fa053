"""The operators where places pass 32 bits, where many routes share a chunk, in
several threads at once, and on streams given for a differentiated call."""

from __future__ import annotations

from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import sort_reference as ref
from gpu_helpers import log
from mixture_experts_expert_mm_amd import moe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def gen(seed, device="cpu"):
    return torch.Generator(device=device).manual_seed(seed)


@pytest.mark.parametrize("T,E,K", [(200000, 7, 4), (300001, 300, 2), (66000, 1024, 16)])
def test_orders_of_many_routes(T, E, K):
    """Chunks of several turns (from 512 x 1024 routes on)."""
    log(f"[large order] T={T} E={E} K={K}")
    ids = torch.randint(-1, E + 1, (T, K), generator=gen(T), dtype=torch.int32)
    rows, o = moe.sort_tokens(torch.arange(T, dtype=F32, device="cuda")[:, None], ids.cuda(), E)
    want = ref.order(ids, E)
    for got, w in zip((o.counts, o.offsets, o.row_of_route, o.route_of_row), want):
        assert torch.equal(got.cpu(), w)
    n = int(want[1][-1])
    assert torch.equal(rows[:n, 0].cpu(), (want[3][:n] // K).float()) and bool((rows[n:] == 0).all())


def test_rows_beyond_32_bits():
    """4.7e9 elements of rows: their last ones come from and go to the right places."""
    T, H, E, K = 82000, 7168, 8, 8
    x = torch.randn(T, H, generator=gen(1, "cuda"), device="cuda", dtype=BF16)
    ids = torch.rand(T, E, generator=gen(2, "cuda"), device="cuda").argsort(1).to(torch.int32)
    rows, o = moe.sort_tokens(x, ids, E)
    assert rows.numel() > 2 ** 32
    at = torch.cat([torch.arange(64, device="cuda"), torch.arange(T * K - 64, T * K, device="cuda"),
                    torch.randint(0, T * K, (256,), generator=gen(3, "cuda"), device="cuda")])
    assert torch.equal(rows[at], x[o.route_of_row[at].long() // K])
    w = torch.full((T, K), 0.125, device="cuda")
    y = moe.combine_tokens(rows, o, w)
    assert torch.equal(y, x)                                   # eight equal parts, exactly
    t = torch.cat([torch.arange(8, device="cuda"), torch.arange(T - 8, T, device="cuda")])
    drows, dw = moe.combine_backward(x, rows, o, w)
    assert torch.equal(drows[at], (x[o.route_of_row[at].long() // K].float() * 0.125).to(BF16))
    want = x[t].double().square().sum(1)[:, None].expand(-1, K)
    assert bool(((dw[t].double() - want).abs() <= 2 * H * ref.U32 * want).all())
    del rows, drows, y


def test_activation_beyond_32_bits():
    M, I = 530000, 4096
    h = torch.randn(M, 2 * I, generator=gen(4, "cuda"), device="cuda", dtype=BF16)
    assert h.numel() > 2 ** 32
    a, q, s = moe.swiglu_forward(h)
    da = torch.ones_like(a)
    dh = moe.swiglu_backward(da, q, s)
    for at in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        part = h[at].contiguous()
        b, p, r = moe.swiglu_forward(part)
        assert torch.equal(a[at], b) and torch.equal(q[at], p) and torch.equal(s[at], r)
        assert torch.equal(dh[at], moe.swiglu_backward(da[at].contiguous(), p, r))


@pytest.mark.parametrize("M,N,K,G", [(300000, 8192, 128, 1), (600000, 256, 8192, 1), (900, 8192, 8192, 66)])
def test_products_beyond_32_bits(M, N, K, G):
    """More than 2^31 outputs, 2^32 codes, 2^32 weights."""
    log(f"[large product] M={M} N={N} K={K} G={G}")
    g = gen(M, "cuda")
    draw = lambda *shape: torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)
    q, w = draw(M, K), draw(G, N, K)
    s, ws = torch.rand(M, generator=g, device="cuda"), torch.rand(G, N, generator=g, device="cuda")
    per = -(-M // G)
    off = torch.arange(0, G, dtype=torch.int32, device="cuda") * per
    cnt = (M - off).clamp(0, per).to(torch.int32)
    y = moe.int8_matmul(q, s, w if G > 1 else w[0], ws if G > 1 else ws[0], *((off, cnt) if G > 1 else ()))
    for at in (0, M // 2, M - 20):
        rows = torch.arange(at, at + 20, device="cuda")
        for r in rows[[0, 7, 19]].tolist():
            e = r // per
            acc = (w[e].double() @ q[r].double())
            want = acc * ws[e].double() * s[r].double()
            assert bool(((y[r].double() - want).abs() <= want.abs() * (3 * ref.U32 + ref.HALF[BF16]) * 1.01).all())


def test_several_threads():
    """Calls from several threads, each on a stream of its own, with plans that they make at the same time."""
    E, K, H, I = 6, 3, 64, 128
    w = torch.randint(-100, 100, (E, 2 * I, H), dtype=torch.int8, device="cuda")
    ws = torch.rand(E, 2 * I, device="cuda")

    def step(T, stream):
        x = torch.randn(T, H, generator=gen(T)).to(BF16).cuda()
        ids = torch.randint(0, E, (T, K), generator=gen(T), dtype=torch.int32).cuda()
        torch.cuda.current_stream().synchronize()
        out = []
        for _ in range(5):
            rows, o = moe.sort_tokens(x, ids, E, stream=stream)
            a = moe.swiglu(moe.int8_linear(rows, w, ws, o.offsets, o.counts, stream=stream), stream=stream)
            out.append(moe.combine_tokens(a, o, stream=stream))
        stream.synchronize()
        return [t.cpu() for t in out]

    sizes = [5, 700, 64, 1900, 333, 2100]
    want = [step(T, torch.cuda.default_stream()) for T in sizes]
    with ThreadPoolExecutor(len(sizes)) as pool:
        got = list(pool.map(lambda T: step(T, torch.cuda.Stream()), sizes))
    for a, b in zip(got, want):
        assert all(torch.equal(x, b[0]) for x in a + b)


def test_gradients_on_a_given_stream():
    """The backward pass of a call on a given stream, asked for on another one."""
    T, H, E, K = 3000, 256, 8, 4
    x = torch.randn(T, H, generator=gen(1)).cuda()
    ids = torch.randint(0, E, (T, K), generator=gen(2), dtype=torch.int32).cuda()
    w = torch.rand(T, K, generator=gen(3)).cuda()
    dy = torch.randn(T, H // 2, generator=gen(4)).cuda()

    def step(x, w, **kw):
        rows, o = moe.sort_tokens(x, ids, E, **kw)
        return moe.combine_tokens(moe.swiglu(rows, **kw), o, w, **kw)

    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    want = torch.autograd.grad(step(xr, wr), (xr, wr), dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        y = step(xr, wr, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        got = torch.autograd.grad(y, (xr, wr), dy)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
