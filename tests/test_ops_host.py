"""Host side of the router, the few-token layer and the block-scaled product
(no GPU): plans, their limits, and refusals before any HIP call."""

import ctypes
import os

import pytest
import torch

from mixture_experts_expert_mm_amd import binding as B
from mixture_experts_expert_mm_amd import moe

GOOD = 1 << 20          # an aligned fake address; never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.lib_path()):
        from mixture_experts_expert_mm_amd import _build
        _build.build()
    return B.load()


def test_struct_sizes():
    assert ctypes.sizeof(B.MMRouterProblem) == 48 and ctypes.sizeof(B.MMRouterPlan) == 48 + 8 + 8 + 32
    assert ctypes.sizeof(B.MMFewProblem) == 64 and ctypes.sizeof(B.MMFewPlan) == 64 + 8 + 8 + 32
    assert ctypes.sizeof(B.MMBlockProblem) == 32 and ctypes.sizeof(B.MMBlockPlan) == 32 + 8 + 8 + 32


def refused(fn, *a, status=1, **kw):
    with pytest.raises(B.MMError) as ei:
        fn(*a, **kw)
    assert ei.value.status == status


@pytest.mark.parametrize("dims", [(0, 256, 8, 2), (1 << 25, 256, 8, 2), (4, 100, 8, 2), (4, 128, 8, 2), (4, 256, 0, 1),
                                  (4, 256, 1025, 2), (4, 256, 8, 0), (4, 256, 8, 9), (4, 256, 128, 65), (4, 16640, 8, 2)])
def test_router_plan_refuses(dims):
    refused(B.mm_router_plan_create, *dims)


def test_router_plan():
    refused(B.mm_router_plan_create, 4, 256, 8, 2, 5, status=2)
    refused(B.mm_router_plan_create, 4, 256, 8, 2, route_scale=float("nan"))
    refused(B.mm_router_plan_create, 4, 256, 8, 2, renormalize=3)
    p = B.mm_router_plan_create(16384, 7168, 256, 8)
    assert p.workspace_bytes >= 16384 * 256 * 4
    assert B.mm_router_plan_create(1, 256, 1, 1).workspace_bytes > 0


@pytest.mark.parametrize("dims", [(0, 256, 128, 8, 2), (65, 256, 128, 8, 2), (4, 300, 128, 8, 2), (4, 256, 100, 8, 2),
                                  (4, 256, 128, 0, 1), (4, 256, 128, 1025, 2), (4, 256, 128, 8, 9),
                                  (4, 256, 128, 64, 33)])
def test_few_plan_refuses(dims):
    refused(B.mm_few_plan_create, *dims)


def test_few_plan():
    refused(B.mm_few_plan_create, 4, 256, 128, 8, 2, 3, status=2)
    refused(B.mm_few_plan_create, 4, 256, 128, 8, 2, y_dtype=7, status=2)
    refused(B.mm_few_plan_create, 4, 256, 128, 8, 2, num_shared_experts=2)
    refused(B.mm_few_plan_create, 4, 256, 128, 1024, 2, num_shared_experts=1)
    refused(B.mm_few_plan_create, 4, 256, 128, 8, 2, activation_clamp=-1.0)
    refused(B.mm_few_plan_create, 4, 256, 128, 8, 2, activation_clamp=float("nan"))
    a = B.mm_few_plan_create(64, 256, 128, 64, 32, num_shared_experts=1)
    assert a.workspace_bytes >= 64 * 33 * 128 * 2
    assert B.mm_few_plan_create(64, 256, 128, 64, 32, y_dtype="f32").workspace_bytes >= 3 * 64 * 32 * 128 * 2


@pytest.mark.parametrize("dims", [(0, 16, 128, 1), (4, 0, 128, 1), (4, 24, 128, 1), (4, 16, 100, 1), (4, 16, 128, 0),
                                  (4, 16, 128, 1025), (1 << 25, 16, 128, 1), (4, 1 << 21, 128, 1), (4, 16, 1 << 21, 1)])
def test_block_plan_refuses(dims):
    refused(B.mm_block_plan_create, *dims)


def test_entry_points_validate_before_any_hip_call(lib):
    P = ctypes.byref
    rp = B.mm_router_plan_create(4, 256, 8, 2)
    args = [P(rp), GOOD, GOOD, None, None, GOOD, GOOD, GOOD, 1 << 40, None]

    def call(fn, args, i, v):
        a = list(args)
        a[i] = v
        return fn(*a)

    for i in (1, 2, 5, 6, 7):
        assert call(lib.mm_router, args, i, None) == 1
        assert call(lib.mm_router, args, i, GOOD + 2) == 1
    assert call(lib.mm_router, args, 3, GOOD + 2) == 1
    assert call(lib.mm_router, args, 8, 16) == 3
    bad = B.MMRouterPlan.from_buffer_copy(rp)
    bad.prob.num_topk = 3
    assert call(lib.mm_router, args, 0, P(bad)) == 1
    assert call(lib.mm_router, args, 0, None) == 1

    fp = B.mm_few_plan_create(4, 256, 128, 8, 2, "fp8")
    args = [P(fp), GOOD, GOOD, GOOD, None, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, 1 << 40, None]
    for i in (1, 2, 3, 5, 6, 7, 8, 9, 10):
        assert call(lib.mm_moe_few, args, i, None) == 1
        assert call(lib.mm_moe_few, args, i, GOOD + 2) == 1
    assert call(lib.mm_moe_few, args, 11, 16) == 3
    bad = B.MMFewPlan.from_buffer_copy(fp)
    bad.workspace_bytes = 0
    assert call(lib.mm_moe_few, args, 0, P(bad)) == 1

    for a in ([0, 128], [4, 0], [4, 100], [1 << 25, 128], [4, 1 << 21]):
        assert lib.mm_block_quantize(*a, GOOD, GOOD, GOOD, None) == 1
    for bad in ([None, GOOD, GOOD], [GOOD, None, GOOD], [GOOD, GOOD, None], [GOOD + 8, GOOD, GOOD]):
        assert lib.mm_block_quantize(4, 128, *bad, None) == 1

    bp = B.mm_block_plan_create(4, 16, 128)
    args = [P(bp), GOOD, GOOD, GOOD, GOOD, None, None, GOOD, None]
    for i in (1, 2, 3, 4, 7):
        assert call(lib.mm_block_gemm, args, i, None) == 1
        assert call(lib.mm_block_gemm, args, i, GOOD + 2) == 1
    assert call(lib.mm_block_gemm, args, 5, GOOD) == 1           # one group array without the other
    assert call(lib.mm_block_gemm, args, 6, GOOD) == 1
    gp = B.mm_block_plan_create(4, 16, 128, 3)
    assert call(lib.mm_block_gemm, args, 0, P(gp)) == 1           # several groups need their rows
    args = [P(bp), GOOD, GOOD, GOOD, None, None, GOOD, GOOD, 1 << 40, None]
    for i in (1, 2, 3, 6, 7):
        assert call(lib.mm_block_linear, args, i, None) == 1
    assert call(lib.mm_block_linear, args, 8, 16) == 3
    assert call(lib.mm_block_linear, args, 4, GOOD) == 1


def test_functions_refuse_host_tensors_and_wrong_shapes():
    bf = dict(dtype=torch.bfloat16)
    x = torch.zeros(2, 256, **bf)
    with pytest.raises(ValueError, match="on a GPU"):
        moe.route(x, torch.zeros(8, 256, **bf), topk=2)
    with pytest.raises(ValueError, match="a matrix"):
        moe.route(x[0], torch.zeros(8, 256, **bf), topk=2)
    with pytest.raises(ValueError, match="on a GPU"):
        moe.moe_few(x, None, None)
    with pytest.raises(ValueError, match="on a GPU"):
        moe.block_quantize(x)
    with pytest.raises(ValueError, match="on a GPU"):
        moe.block_linear(x, None, None)
    with pytest.raises(ValueError, match="a matrix"):
        moe.block_matmul(None, None, None, None)
    m = x[:, ::2]
    with pytest.raises(ValueError, match="not contiguous"):
        moe._need("x", m, torch.bfloat16, (2, 128), m.device)
    with pytest.raises(ValueError, match="bfloat16"):
        moe._need("x", x, torch.float32, (2, 256), x.device)
    g = torch.zeros(2, 256, requires_grad=True, **bf)
    with pytest.raises(ValueError, match="gradient"):
        moe._need("x", g, torch.bfloat16, (2, 256), g.device)
    with torch.no_grad():
        moe._need("x", g, torch.bfloat16, (2, 256), g.device)


def test_kernel_names():
    assert [B.mm_kernel_name(i) for i in range(10, 16)] == ["router", "router_select", "few_l1", "few_l2",
                                                          "block_quantize", "block_gemm"]
    assert B.mm_kernel_name(16) == "unknown"
