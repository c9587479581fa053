"""Raw stream handles: 0 is the default stream, anything else the stream that it belongs to."""

from __future__ import annotations

import pytest
import torch

from mixture_experts_expert_mm_amd import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("current", ["default", "side"])
def test_handles_name_the_streams_they_belong_to(current):
    dev = torch.device("cuda", torch.cuda.current_device())
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(other if current == "side" else torch.cuda.default_stream(dev)):
        for handle in (torch.cuda.default_stream(dev).cuda_stream, side.cuda_stream, other.cuda_stream):
            with moe._stream_of(dev, handle):
                assert torch.cuda.current_stream(dev).cuda_stream == handle
                assert moe._raw_stream(dev) == handle


def test_default_stream_by_its_handle_keeps_the_order():
    """Producer, operator and consumer on the default stream, without a wait between them."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4096, 2048, generator=g).to(torch.bfloat16).cuda()
    want = moe.block_quantize(x)
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    buf = torch.zeros_like(x)
    handle = torch.cuda.default_stream().cuda_stream
    for _ in range(5):
        buf.zero_()
        for _ in range(4):
            big @ big                       # the copy waits behind these
        buf.copy_(x)
        q, s = moe.block_quantize(buf, stream=handle)
        assert torch.equal(s, want[1]) and torch.equal(q.view(torch.uint8), want[0].view(torch.uint8))
