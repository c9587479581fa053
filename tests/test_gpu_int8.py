"""Products of 8-bit integers on the GPU: codes and scales equal to the IEEE
rule's, sums exact, outputs within the roundings of their scaling."""

from __future__ import annotations

import pytest
import torch

import swiglu_reference as ref
from gpu_helpers import log
from mixture_experts_expert_mm_amd import moe
from sort_reference import F64, HALF, TINY, U32

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = {"bf16": BF16, "f16": F16, "f32": F32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def codes(seed, *shape):
    return torch.randint(-128, 128, shape, generator=gen(seed), dtype=torch.int8)


def scales(seed, *shape):
    return torch.rand(*shape, generator=gen(seed)) * 0.01 + 1e-4


def exact(q, s, w, ws, dt):
    """y in 64 bits and its error: the sum becomes float32, two float32 products, one rounding."""
    acc = q.to(F64) @ w.to(F64).t()          # whole numbers below 2^53
    y = acc * ws.to(F64) * s.to(F64)[:, None]
    return y, y.abs() * (3 * U32 + HALF[dt]) * 1.01 + TINY[dt]


def within(y, want, err, what=""):
    y = y.detach().cpu().to(F64)
    over = (y - want).abs() - err
    assert y.shape == want.shape and bool((over <= 0).all()), (what, float(over.max()), (over > 0).nonzero()[:4])


# every kernel (up to 8 rows; tiles of 32 x 32, 64 x 32, 64 x 64, 128 x 64, 128 x 128 for one round and two, 256 x 256 with a
# rest of 1, 16, 17, 128, 129 and 255 rows), K of less than a step, with a last step of every length, an even and an odd
# number of steps
SHAPES = [(1, 1, 16), (1, 7168, 2048), (3, 5, 48), (16, 40, 144), (16, 1000, 7168), (17, 16, 128), (17, 33, 272), (31, 1001, 400),
          (64, 512, 1008), (65, 130, 640), (100, 4096, 272), (200, 1026, 896), (129, 4100, 1152), (300, 2048, 64), (512, 2052, 2064),
          (1100, 4096, 336), (2049, 2052, 400), (2064, 1999, 1280), (2065, 2048, 144), (2176, 2050, 640), (2177, 2048, 656),
          (2303, 2111, 128), (4097, 1024, 1408), (40, 150, 8192), (24, 3, 131056),
          (2049, 4100, 400), (2064, 4099, 272), (2065, 4096, 144), (2176, 4098, 640), (2177, 4096, 656), (2303, 4223, 128), (2304, 4352, 48),
          (600, 3500, 272), (1000, 2100, 528)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("y_dtype", ["bf16", "f16", "f32"])
def test_product(M, N, K, y_dtype):
    log(f"[int8] M={M} N={N} K={K} {y_dtype}")
    q, w, s, ws = codes(M, M, K), codes(N + 1, N, K), scales(K, M), scales(K + 1, N)
    if y_dtype == "f16":
        s = s * 1e-2                          # inside float16's range
    y = moe.int8_matmul(q.cuda(), s.cuda(), w.cuda(), ws.cuda(), y_dtype=y_dtype)
    assert y.dtype == TYPES[y_dtype]
    within(y, *exact(q, s, w, ws, TYPES[y_dtype]))


@pytest.mark.parametrize("M,K", [(2, 131056), (20, 131056), (300, 131056)])
def test_largest_sums(M, K):
    """Codes of -128 throughout: 131056 * 2^14, the largest sum that int32 takes."""
    q, w = torch.full((M, K), -128, dtype=torch.int8), torch.full((40, K), -128, dtype=torch.int8)
    w[1::2] = 127
    one = torch.ones(40)
    y = moe.int8_matmul(q.cuda(), torch.ones(M).cuda(), w.cuda(), one.cuda(), y_dtype="f32").cpu()
    assert bool((y[:, ::2] == float(K * 16384)).all()) and bool((y[:, 1::2] == float(torch.tensor(-K * 16256, dtype=F32))).all())


@pytest.mark.parametrize("x_dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 7168), (5, 1616), (4, 2048), (16, 512), (300, 4096), (37, 4112), (9, 16384), (3, 16400), (2, 131056)])
def test_quantize_and_linear(x_dtype, M, K):
    log(f"[int8 linear] M={M} K={K} {x_dtype}")
    x = torch.randn(M, K, generator=gen(M + K)) * torch.exp(torch.randn(M, 1, generator=gen(K)))
    x[0, :8] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, 127.0, -127.0, 63.5])   # ties, where the scale is 1
    x[0, 8:] = x[0, 8:].clamp(-100, 100).round()
    if M > 2:
        x[1] = 0                              # a row of zeros: the smallest scale
        x[2] *= 1e-6
    x = x.to(x_dtype)
    wq, wsc = ref.codes(x)
    q, s = moe.int8_quantize(x.cuda())
    assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), wsc)
    w, ws = codes(3, 50, K), scales(4, 50) * 1e-3
    for y_dtype in ("bf16", "f32"):
        y = moe.int8_linear(x.cuda(), w.cuda(), ws.cuda(), y_dtype=y_dtype)
        assert torch.equal(y, moe.int8_matmul(q, s, w.cuda(), ws.cuda(), y_dtype=y_dtype))
        within(y, *exact(wq, wsc, w, ws, TYPES[y_dtype]))


@pytest.mark.parametrize("M", [3, 40])
def test_rows_that_are_no_numbers(M):
    x = torch.randn(M, 256, generator=gen(1)).to(BF16)
    x[0, 3], x[1, 255], x[2, 0] = float("nan"), float("inf"), -float("inf")
    w, ws = codes(3, 70, 256), scales(4, 70)
    y = moe.int8_linear(x.cuda(), w.cuda(), ws.cuda())
    assert bool(y[:3].isnan().all()) and bool(y[3:].isfinite().all())
    q, s = moe.int8_quantize(x.cuda())
    assert bool((q[:3] == 0).all()) and bool(s[0].isnan()) and bool(s[1:3].isinf().all())


def groups_of(G, M, seed, kind):
    """offsets and counts of groups in order, with gaps, empty ones, and one that reaches beyond the rows."""
    g = gen(seed)
    cut = torch.sort(torch.randint(0, M + 1, (G - 1,), generator=g))[0].tolist()
    ends = cut + [M]
    off, cnt, lo = [], [], 0
    for i, e in enumerate(ends):
        gap = 1 if kind == "gaps" and e - lo > 3 else 0
        off.append(lo + gap)
        cnt.append(e - lo - gap)
        lo = e
    if kind == "gaps":
        cnt[-1] += 7                          # clipped at the last row
    return torch.tensor(off, dtype=torch.int32), torch.tensor(cnt, dtype=torch.int32)


@pytest.mark.parametrize("G,M,N,K", [(2, 9, 40, 144), (5, 100, 130, 272), (32, 64, 256, 640), (3, 700, 516, 1008), (8, 1500, 2049, 400),
                                     (70, 3000, 256, 256), (4, 5000, 1024, 912), (300, 40, 64, 128), (33, 9000, 512, 384),
                                     (40, 6000, 1024, 272), (9, 20000, 641, 144)])
@pytest.mark.parametrize("kind", ["dense", "gaps"])
def test_groups(G, M, N, K, kind):
    log(f"[int8 groups] G={G} M={M} N={N} K={K} {kind}")
    q, w, s, ws = codes(M, M, K), codes(N, G, N, K), scales(K, M), scales(K + 1, G, N)
    off, cnt = groups_of(G, M, M + G, kind)
    mark = torch.full((M, N), 7.0, dtype=BF16).cuda()
    y = moe.int8_matmul(q.cuda(), s.cuda(), w.cuda(), ws.cuda(), off.cuda(), cnt.cuda(), y=mark)
    assert y is mark
    want, err = torch.full((M, N), 7.0, dtype=F64), torch.zeros(M, N, dtype=F64)
    for i in range(G):
        lo, hi = int(off[i]), min(M, int(off[i] + cnt[i]))
        if lo < hi:
            want[lo:hi], err[lo:hi] = exact(q[lo:hi], s[lo:hi], w[i], ws[i], BF16)
    within(y, want, err)
    x = torch.randn(M, K, generator=gen(G)).to(BF16)
    qx, sx = moe.int8_quantize(x.cuda())
    offs = torch.cat([off, torch.tensor([M], dtype=torch.int32)]).cuda()       # G + 1 offsets do too
    a = moe.int8_linear(x.cuda(), w.cuda(), ws.cuda(), offs, cnt.cuda(), y=torch.zeros(M, N, dtype=BF16, device="cuda"))
    b = moe.int8_matmul(qx, sx, w.cuda(), ws.cuda(), off.cuda(), cnt.cuda(), y=torch.zeros(M, N, dtype=BF16, device="cuda"))
    assert torch.equal(a, b)


def test_one_group_of_some_rows():
    """One matrix over a part of the rows; the others are left as they are."""
    q, w, s, ws = codes(1, 600, 256), codes(2, 1, 300, 256), scales(3, 600), scales(4, 1, 300)
    for lo, n in ((0, 600), (5, 0), (17, 300), (599, 1), (600, 4), (-3, 10)):
        y = torch.full((600, 300), 2.0, device="cuda")
        moe.int8_matmul(q.cuda(), s.cuda(), w.cuda(), ws.cuda(), torch.tensor([lo], dtype=torch.int32).cuda(),
                        torch.tensor([n], dtype=torch.int32).cuda(), y_dtype="f32", y=y)
        a, b = max(lo, 0), min(600, lo + n)
        want, err = torch.full((600, 300), 2.0, dtype=F64), torch.zeros(600, 300, dtype=F64)
        if a < b:
            want[a:b], err[a:b] = exact(q[a:b], s[a:b], w[0], ws[0], F32)
        within(y, want, err, (lo, n))


def test_empty_streams_and_graphs():
    w, ws = codes(2, 130, 384).cuda(), scales(4, 130).cuda()
    assert moe.int8_linear(torch.zeros(0, 384, device="cuda"), w, ws).shape == (0, 130)
    assert moe.int8_quantize(torch.zeros(0, 384, device="cuda"))[0].shape == (0, 384)
    for M in (2, 70, 1200):
        xs = [torch.randn(M, 384, generator=gen(i)).to(BF16).cuda() for i in range(3)]
        want = [moe.int8_linear(x, w, ws) for x in xs]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        got = moe.int8_linear(xs[1], w, ws, stream=st)
        st.synchronize()
        assert torch.equal(got, want[1])
        xb = xs[0].clone()
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = moe.int8_linear(xb, w, ws)
            graphs.append((graph, y))
        for i in range(3):
            for graph, y in graphs:
                xb.copy_(xs[i])
                graph.replay()
                moe.int8_linear(xs[2 - i], w, ws)
                torch.cuda.synchronize()
                assert torch.equal(y, want[i])
