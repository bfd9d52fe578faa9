"""The block's balance loss on a stream of its own."""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe
import synth

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the block on a stream of its own
def test_block_made_while_its_stream_is_busy():
    """A block made on a busy stream and used on another at once: its own constants are there."""
    shape = synth.WORKLOADS["tiny"].with_(T=64, H=256, E=16, K=4, I=128, I_shared=0)
    w = synth.make_weights(shape, device="cuda", seed=0, std=0.05)
    router = synth.make_router(shape, device="cuda", seed=0, std=0.05)
    nw = torch.ones(shape.H, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dout = (torch.randn((shape.T, shape.H), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    got = []
    torch.cuda.synchronize()
    for busy in (False, True):
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(s1):
            old = [torch.full((1,), 9.0, device="cuda") for _ in range(256)]  # what the block's memory holds before
            s1.synchronize()
            del old
            if busy:
                torch.cuda._sleep(200_000_000)  # about 0.1 s
            block = moe.MoEBlock(shape, w, router, nw, balance_coef=0.5)
        block.forward(x, stream=s2)
        block.backward(dout, stream=s2)
        s2.synchronize()
        got.append(block.dlogits.clone())
        torch.cuda.synchronize()
    assert torch.equal(got[0], got[1])
