"""The activation, its 8-bit copy and its gradient on the GPU against plain
64-bit implementations."""

from __future__ import annotations

import math

import pytest
import torch

import swiglu_reference as ref
from gpu_helpers import log
from mixture_experts_expert_mm_amd import moe

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(y, want, err):
    over = (y.detach().cpu().to(F64) - want).abs() - err
    assert bool((over <= 0).all()), (float(over.max()), float(want.abs().max()))


def inputs(M, I, dtype, seed=0):
    g = gen(seed + M + I)
    h = torch.randn(M, 2 * I, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    h[::5, : min(I, 130)] = 0                                   # groups of zeros, and half of them
    if M > 2:
        h[2] *= 2.0 ** -20                                      # scales at the floor
        h[1] *= 20
    return h.to(dtype), torch.randn(M, I, generator=g).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,I", [(1, 1), (1, 8), (3, 127), (5, 128), (2, 129), (7, 136), (17, 250), (64, 1408), (333, 2048),
                                 (1, 16384), (2000, 33), (4099, 24)])
@pytest.mark.parametrize("clamp", [None, 1.5, 0.0])
def test_forward_copy_and_gradient(M, I, dtype, clamp):
    log(f"[swiglu] M={M} I={I} {dtype} clamp={clamp}")
    h, da = inputs(M, I, dtype)
    a, q, s = moe.swiglu_forward(h.cuda(), activation_clamp=clamp)
    within(a, *ref.forward(h, clamp))
    wq, ws = ref.keep(h)
    assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), ws)
    assert torch.equal(moe.swiglu(h.cuda(), activation_clamp=clamp), a)
    dh = moe.swiglu_backward(da.cuda(), q, s, activation_clamp=clamp)
    within(dh, *ref.backward(da, wq, ws, clamp))
    hr = h.cuda().requires_grad_()
    y = moe.swiglu(hr, activation_clamp=clamp)
    y.backward(da.cuda())
    assert torch.equal(y.detach(), a) and torch.equal(hr.grad, dh)


def test_gradient_against_differences():
    """The gradient is that of the activation at the kept values: there, differences of the forward pass agree."""
    h, da = inputs(6, 300, F32, 3)
    q, s = ref.keep(h)
    v = ref.kept(q, s)
    dh = moe.swiglu_backward(da.cuda(), q.cuda(), s.cuda()).cpu().to(F64)
    step = 2.0 ** -10
    for seed in range(4):
        d = torch.randn(v.shape, generator=gen(seed)).to(F64)
        up, down = ref.forward((v.to(F64) + step * d).float())[0], ref.forward((v.to(F64) - step * d).float())[0]
        slope = ((up - down) * da.to(F64)).sum() / (2 * step)
        # rounding v +- step d to float32 (half a step of |v|, times a slope of at most 1.1 |u| + |g|), and the third
        # derivative: below (|u| + 1) |d|^3
        g, u, w = v[:, :300].abs().to(F64), v[:, 300:].abs().to(F64), da.abs().to(F64)
        rest = (w * ((1.1 * u + g) * (u + g) * 2 ** -24 / step)).sum() + step ** 2 * (w * (u + 1) * d.abs().amax() ** 3).sum()
        assert abs(float(slope - (dh * d).sum())) <= float(rest)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_special_values(dtype):
    """NaN and infinities stay in their places of a, and in their groups of the copy and the gradient."""
    h, da = inputs(4, 300, dtype, 9)
    h[0, 5] = float("nan")
    h[1, 300 + 140] = float("inf")
    h[2, 299] = -float("inf")
    h[3, 7], h[3, 8] = 200.0, -200.0                            # e^200 is beyond float32
    for clamp in (None, 2.0):
        a, q, s = moe.swiglu_forward(h.cuda(), activation_clamp=clamp)
        dh = moe.swiglu_backward(da.cuda(), q, s, activation_clamp=clamp)
        a, q, s, dh = a.cpu().float(), q.cpu(), s.cpu(), dh.cpu().float()
        assert math.isnan(a[0, 5]) and int(a[0].isnan().sum()) == 1
        assert bool(a[1].isfinite().all()) == (clamp is not None)
        fine, _ = ref.forward(h[3:], clamp)
        assert torch.allclose(a[3:].to(F64), fine, rtol=2.0 ** -7, atol=2.0 ** -20) and bool(a[3].isfinite().all())
        n = 3
        assert math.isnan(s[0, 0]) and math.isinf(s[1, n + 1]) and math.isinf(s[2, 2])
        assert bool((q[0, :128] == 0).all()) and bool((q[1, 300 + 128:300 + 256] == 0).all()) and bool((q[2, 256:300] == 0).all())
        bad = dh.isnan()
        # the gate's gradient reads both halves, the up half's only the gate
        for row, lo, hi in ((0, 0, 128), (1, 128, 256), (2, 256, 300)):
            want = torch.zeros(600, dtype=torch.bool)
            want[lo:hi] = want[300 + lo:300 + hi] = True
            inside = ~(ref.kept(q, s)[row].abs() > ref.clamp_of(clamp))       # elsewhere the gradient is 0
            assert torch.equal(bad[row, lo:hi], inside[lo:hi])
            assert torch.equal(bad[row, 300 + lo:300 + hi], inside[300 + lo:300 + hi] & (row != 1))
            assert not bool(bad[row][~want].any())
        assert not bool(bad[3].any())


def test_gradient_shapes_streams_and_graphs():
    h, da = inputs(40, 96, BF16, 4)
    want = moe.swiglu_backward(torch.ones_like(da).cuda(), *moe.swiglu_forward(h.cuda())[1:])
    hr = h.cuda().requires_grad_()
    moe.swiglu(hr).sum().backward()                             # an expanded gradient
    assert torch.equal(hr.grad, want)
    buf = torch.cat([torch.zeros(1), da.flatten().float()]).to(BF16).cuda()
    a, q, s = moe.swiglu_forward(h.cuda())
    want = moe.swiglu_backward(da.cuda(), q, s)
    for d in (buf[1:].view(40, 96), da.t().contiguous().cuda().t()):     # an odd address, a transposed one
        hr = h.cuda().requires_grad_()
        moe.swiglu(hr).backward(d)
        assert torch.equal(hr.grad, want)
    e = torch.zeros(0, 8, device="cuda", requires_grad=True)
    moe.swiglu(e).sum().backward()
    assert e.grad.shape == (0, 8)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = moe.swiglu(h.cuda(), stream=st)
    st.synchronize()
    assert torch.equal(got, a)
    hb, db = h.cuda(), da.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.swiglu_forward(hb)
        dh = moe.swiglu_backward(db, *out[1:])
        with pytest.raises(RuntimeError, match="capture"):
            moe.swiglu(hr)
    for seed in range(3):
        h2, d2 = inputs(40, 96, BF16, 50 + seed)
        hb.copy_(h2)
        db.copy_(d2)
        graph.replay()
        want = moe.swiglu_forward(hb)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert torch.equal(dh, moe.swiglu_backward(db, *want[1:]))


def alternate(t, I, g):
    """Columns [gate | up] of t in turns of g."""
    return t.view(t.shape[0], 2, I // g, g).transpose(1, 2).reshape(t.shape).contiguous()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,I,g", [(1, 32, 32), (5, 128, 32), (3, 8, 8), (40, 200, 40), (333, 1408, 32), (17, 2048, 32), (9, 264, 8),
                                   (4, 264, 264), (700, 96, 24)])
@pytest.mark.parametrize("clamp", [None, 1.5])
def test_alternating_columns(M, I, g, dtype, clamp):
    """The same values, codes, scales and gradients wherever the columns lie."""
    h, da = inputs(M, I, dtype, 7)
    a, q, s = moe.swiglu_forward(h.cuda(), activation_clamp=clamp)
    dh = moe.swiglu_backward(da.cuda(), q, s, activation_clamp=clamp)
    turned = alternate(h, I, g).cuda()
    b, p, r = moe.swiglu_forward(turned, activation_clamp=clamp, gate_up_group=g)
    assert torch.equal(a, b) and torch.equal(s, r) and torch.equal(alternate(q, I, g), p)
    assert torch.equal(moe.swiglu(turned, activation_clamp=clamp, gate_up_group=g), a)
    d = moe.swiglu_backward(da.cuda(), p, r, activation_clamp=clamp, gate_up_group=g)
    assert torch.equal(alternate(dh, I, g), d)
    hr = turned.requires_grad_()
    moe.swiglu(hr, activation_clamp=clamp, gate_up_group=g).backward(da.cuda())
    assert torch.equal(hr.grad, d)
