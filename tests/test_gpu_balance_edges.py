"""The balance loss of the smallest scores, for every number of experts in its two-launch form, and the block's on a
stream of its own."""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe
import synth
from test_gpu_balance import F64, I32, SCORES, grad64, problem, reference, run, share_tol, shares64

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


# ---------------------------------------------------------------- shapes of the two-launch form
# More logits than one launch takes (2^14 or 2^16 per thread block of a cluster), for each number of lanes and values.
STRIPS = [(100000, 8, 2, 1), (100000, 7, 2, 3), (20000, 16, 3, 1), (60000, 13, 3, 3), (30000, 32, 4, 1), (30000, 30, 4, 2),
          (9000, 64, 4, 1), (9000, 63, 4, 2), (5000, 120, 8, 2), (5000, 160, 8, 1), (3000, 256, 8, 1), (3000, 250, 8, 2),
          (3000, 255, 8, 1), (2000, 512, 8, 1), (2000, 500, 8, 2), (1500, 1000, 8, 2), (1500, 1024, 32, 1), (1500, 1023, 8, 1)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T, E, K, B", STRIPS)
def test_strips(handle, T, E, K, B, score):
    assert T * E > (1 << (14 if B == 1 else 16)) * 8
    logits, idx, g = problem(T, E, K, seed=T + E)
    ends = [0] + [T * i // B + 3 * i for i in range(1, B)] + [T]
    cfg, seq, counts, prob, loss = run(handle, logits, idx, ends, score, 0.25, E, K)
    rc, rp, rl = reference(logits, idx, ends, score, 0.25, E, K)
    assert torch.equal(counts, rc)
    tol = share_tol(E) + (T / 512 + 64) * 2.0 ** -24  # as test_gpu_balance: a warp's tokens in a row, then warps, strips
    assert ((prob.to(F64) - rp).abs() <= tol * rp).all()
    assert ((loss.to(F64) - rl).abs() <= (tol + (E / 32 + 16) * 2.0 ** -24) * rl).all()
    dloss = torch.rand(B, device="cuda", generator=g) + 0.5
    dl = torch.full((T, E), 7.0, device="cuda")
    moe.balance_loss_backward(handle, cfg, logits, counts, dloss, dl, coef=0.25, score=SCORES[score], seq_offsets=seq)
    want = grad64(logits, counts, ends, dloss, score, 0.25, E, K)
    p = shares64(logits.to(F64), score)
    for b in range(B):
        lo, hi = ends[b], ends[b + 1]
        size = float(dloss[b]) * 0.25 / (hi - lo) * float(counts[b].max()) * E / (K * (hi - lo))
        assert ((dl[lo:hi].to(F64) - want[lo:hi]).abs() <= size * p[lo:hi] * (2 * share_tol(E) + 2.0 ** -20) + 1e-30).all()


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
