"""The router's order and weights where float32 sums go wrong in one direction, beside a NaN, and in runs."""

from __future__ import annotations

import math

import pytest
import torch

import ops_reference as ref
from gpu_helpers import log
from mixture_experts_expert_mm_amd import moe

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64


def drift_case(H, E, per):
    """(x [255, H], w [E, H]): past channel 31 every `per` products add up to just below half an ulp of the running
    sum, which stays near 1, with one sign for expert 6 and the other for expert 4; a float32 sum that rounds as often
    loses them all.  The token's channel 1 raises expert 4 by 1/255 to 255/255 of a little more than what is lost.
    The others' scores are 0."""
    x = torch.zeros(255, H)
    x[:, 0] = 1.0
    x[:, 1] = torch.arange(1, 256) * 2.0 ** -10
    x[:, 32:] = 2.0 ** -12
    small = float(torch.tensor(0.99).to(BF16)) / per * 2.0 ** -12
    step = math.ceil((H - 32) / per / 250)             # of 2^-23: the two lose (H - 32) / per in all
    w = torch.zeros(E, H)
    w[6, 0] = w[4, 0] = 1.0
    w[4, 1] = step * 2.0 ** -13
    w[6, 32:], w[4, 32:] = small, -small
    return x.to(BF16), w.to(BF16)


@pytest.mark.parametrize("H", [1024, 7168, 16384])
@pytest.mark.parametrize("T,E", [(1, 8), (255, 40), (3000, 40), (2000, 128), (16384, 256), (20000, 66), (33000, 66), (9000, 600)])
@pytest.mark.parametrize("per", [8, 32])
def test_router_order_of_sums_that_drift(T, E, H, per):
    """One slice of the hidden dimension or several, small and large tiles: the same order as in 64 bits."""
    log(f"[router drift] T={T} H={H} E={E} {per}")
    x, w = drift_case(H, E, per)
    z = x.to(F64) @ w.to(F64).t()
    want = z.sort(dim=1, descending=True, stable=True)[1][:, :2].to(torch.int32)
    assert 0 < int((want[:, 0] == 6).sum()) < 255
    at = torch.arange(T) * 97 % 255
    if T == 1:
        at = (want[:, 0] == 6).nonzero()[-1]           # the closest one
    xd = x.cuda()[at.cuda()].contiguous()
    ids, _ = moe.route(xd, w.cuda(), topk=2)
    assert torch.equal(ids.cpu(), want[at]), (ids.cpu() != want[at]).any(1).sum()


@pytest.mark.parametrize("T,E", [(200, 40), (3000, 40), (2000, 128), (33000, 66), (9000, 600)])
@pytest.mark.parametrize("sums", [1.0, -1.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_router_order_of_sums_that_drift_beside_a_nan(T, E, sums, sign):
    """The same with sums of either sign, and a NaN in the weights of the expert between the two, which says nothing
    of them (every other expert is switched off)."""
    log(f"[router drift nan] T={T} E={E} {sums} {sign}")
    x, w = drift_case(7168, E, 8)
    w *= sums
    z = x.to(F64) @ w[[4, 6]].to(F64).t()
    want = torch.where(z[:, 1] > z[:, 0], 6, 4).to(torch.int32)
    w[5, 3], w[5, 6000] = math.copysign(math.nan, sign), math.copysign(math.nan, sign)
    bias = torch.full((E,), -math.inf)
    bias[[4, 6]] = 0.0
    at = torch.arange(T) * 97 % 255
    ids, _ = moe.route(x.cuda()[at.cuda()].contiguous(), w.cuda(), bias.cuda(), topk=2, scoring="sigmoid")
    assert torch.equal(ids[:, 0].cpu(), want[at]), (ids[:, 0].cpu() != want[at]).sum()


def cancel_case(T, H, E, seed):
    """Two products of 2^13 that cancel, at both ends of a row: the scores lose their low bits in float32."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(BF16)
    w = (torch.randn(E, H, generator=g) * H ** -0.5).to(BF16)
    x[:, 5], x[:, H - 1] = 1024.0, -1024.0
    w[:, 5] = w[:, H - 1] = 8.0
    return x, w


SIZES = [(5, 7168, 32, 8), (200, 7168, 32, 8), (1500, 2048, 48, 8), (2000, 7168, 128, 8), (600, 16384, 256, 8), (70, 512, 600, 4)]


@pytest.mark.parametrize("T,H,E,K", SIZES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_router_order_beside_a_nan(T, H, E, K, sign):
    """A NaN in one expert's weights leaves the order of the others as the 64-bit scores have it."""
    log(f"[router nan] T={T} H={H} E={E}")
    x, w = cancel_case(T, H, E, 90 + T)
    w[E // 2, 40] = math.copysign(math.nan, sign)
    ids, _ = moe.route(x.cuda(), w.cuda(), topk=K, scoring="sigmoid", renormalize=False)
    want, _, _ = ref.route(x, w, None, K, "sigmoid", False)
    assert torch.equal(ids.cpu(), want), (ids.cpu() != want).any(1).sum()


@pytest.mark.parametrize("T,H,E,K", SIZES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_router_weights_do_not_rise(T, H, E, K, scoring):
    """Experts that only their 64-bit sums tell apart get their weights from the same sums.  A weight is rounded by
    an exponential (2 ulp), a sum and a quotient: two of them are off by 8 * 2^-23 of the value together."""
    log(f"[router weights] T={T} H={H} E={E} {scoring}")
    x, w = cancel_case(T, H, E, 190 + T)
    ids, wts = moe.route(x.cuda(), w.cuda(), topk=K, scoring=scoring, renormalize=False)
    assert torch.equal(ids.cpu(), ref.route(x, w, None, K, scoring, False)[0])
    assert bool((wts[:, 1:] <= wts[:, :-1] * (1 + 8 * 2.0 ** -23)).all())
