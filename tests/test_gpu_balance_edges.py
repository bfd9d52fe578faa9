"""The balance loss of the smallest scores, and the block's on a stream of its own."""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe
import synth
from test_gpu_balance import F64, I32, SCORES, grad64, run, share_tol, shares64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = moe.Handle(0)
    yield h
    torch.cuda.synchronize()
    assert h.device_status() == 0
    h.close()


# ---------------------------------------------------------------- scores that nearly all underflow
@pytest.mark.parametrize("top", [-15.0, -17.0, -18.0, -30.0, -60.0, -69.0, -69.2, -75.0])
def test_small_sigmoid_scores_keep_their_ratios(handle, top):
    """Sigmoid scores whose largest is small, others 18 below it (below the smallest normal number for the last ones):
    each share is as near its value as fp32 exponentials of such logits are. The logits' products with log2 e are rounded
    at up to |x| log2 e: |x| 2^-23 relative at most for each of two scores; then the sum and the quotient."""
    T, E, K = 8, 48, 1
    logits = torch.full((T, E), top - 18.6, device="cuda")
    logits += torch.arange(E, device="cuda") * 2.0 ** -8
    logits[:, 0] = top
    idx = torch.zeros((T, K), dtype=I32, device="cuda")
    cfg, _, counts, prob, _ = run(handle, logits, idx, [0, T], "sigmoid", 1.0, E, K)
    p = shares64(logits.to(F64), "sigmoid")
    tol = 2 * (abs(top) + 20) * 2.0 ** -23 + share_tol(E) + 16 * 2.0 ** -24
    assert ((prob[0].to(F64) - p[0]).abs() <= tol * p[0]).all()
    dl = torch.empty((T, E), device="cuda")
    moe.balance_loss_backward(handle, cfg, logits, counts, torch.ones(1, device="cuda"), dl, score=SCORES["sigmoid"])
    want = grad64(logits, counts, [0, T], [1.0], "sigmoid", 1.0, E, K)
    f = float(counts.max()) * E / (K * T)
    assert ((dl.to(F64) - want).abs() <= 2 * f / T * p * tol).all()


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
