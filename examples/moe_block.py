"""The MoE block trained and served: residual add + RMS norm, gating, experts, and their gradients.

    python examples/moe_block.py            # a GB300; build the library first (see README)

train() fits a block to another block's outputs with plain gradient steps. serve() runs one MXFP8 step the way a
decoder does: the norm writes the router's bf16 rows and the experts' E4M3 codes and E8M0 scales in one pass, and the
layer takes both.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import routed_expert_ffn_04_gb300 as moe  # noqa: E402
import synth  # noqa: E402

SHAPE = synth.WORKLOADS["tiny"].with_(T=256, H=512, E=16, K=4, I=256, I_shared=256)


def make_block(shape, seed, std=0.05):
    w = synth.make_weights(shape, device="cuda", seed=seed, std=std)
    router = synth.make_router(shape, device="cuda", seed=seed, std=std)
    return moe.MoEBlock(shape, w, router, torch.ones(shape.H, dtype=torch.bfloat16, device="cuda"))


def train(steps=60, lr=0.01, shape=SHAPE, seed=0):
    """Mean squared error against a teacher that shares the student's router; returns the losses."""
    teacher, student = make_block(shape, seed), make_block(shape, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    masters = {k: v.float() for k, v in student.w.items()}
    for k, v in masters.items():  # start a little off the teacher
        v += 0.03 * torch.randn(v.shape, device="cuda", generator=g)
        student.w[k].copy_(v)
    x = torch.randn((shape.T, shape.H), device="cuda", generator=g).to(torch.bfloat16)
    res = torch.randn((shape.T, shape.H), device="cuda", generator=g).to(torch.bfloat16)
    want = teacher.forward(x, res)[0].clone()
    losses = []
    for _ in range(steps):
        out, _ = student.forward(x, res)
        err = out.float() - want.float()
        losses.append((err * err).mean())
        grads = student.backward((2.0 / shape.T * err).to(torch.bfloat16))
        for k, v in masters.items():
            v -= lr * grads[k].float()
            student.w[k].copy_(v)
    return torch.stack(losses).tolist()


def serve(shape=synth.WORKLOADS["tiny"].with_(T=64, H=512, E=16, K=4, I=256, I_shared=256, dtype="mxfp8"), seed=0):
    """One MXFP8 step from the residual stream; returns its output, the new stream and the output that the layer
    computes when it quantises the bf16 rows itself."""
    layer = moe.MoELayer(shape, synth.make_weights(shape, device="cuda", seed=seed))
    router = synth.make_router(shape, device="cuda", seed=seed)
    T, H, E, K = shape.T, shape.H, shape.E, shape.K
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    res = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    norm_weight = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    n, q = torch.empty_like(x), torch.empty((T, H), dtype=torch.uint8, device="cuda")
    scale = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    moe.add_rmsnorm(layer.handle, x, norm_weight, 1e-5, residual=res, h_out=res, out=n, q=q, q_scale=scale)
    logits = torch.empty((T, E), device="cuda")
    idx, tw = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    moe.gate_route(layer.handle, layer.cfg, n, router, idx, tw, logits_out=logits)
    out = layer(q, logits, x_scale=scale)
    return out, res, layer(n, logits)


def main():
    losses = train()
    print("training: mean squared error %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
    out, _, inside = serve()
    d = (out.float() - inside.float()).norm() / inside.float().norm()
    print("serving (MXFP8): the norm's codes against the layer's own quantisation of the bf16 rows: %.2e apart" % d)


if __name__ == "__main__":
    main()
