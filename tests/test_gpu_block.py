"""The MoE block (norm, gating, experts, and their gradients together) against automatic differentiation in 64 bits,
in a CUDA graph, and the example that trains and serves it.

Tolerance: a gradient passes through at most about ten roundings to bf16 on its way (n, x_perm, h, dy_perm, dh's
operands, dx_perm, dn, ...), each at most 2^-8 / sqrt(3) = 2.3e-3 rms and independent: 7.2e-3 of the norm; with the
difference that rounded inputs make to gate and up, 2e-2."""
import importlib.util
import os

import pytest
import torch

import routed_expert_ffn_04_gb300 as moe
import synth

pytestmark = pytest.mark.gpu
BF, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load(build_if_missing=True)


def _block(shape, rt, seed=0):
    w = synth.make_weights(shape, device="cuda", seed=seed, std=0.05)
    router = synth.make_router(shape, device="cuda", seed=seed, std=0.05)
    nw = (1 + 0.1 * torch.randn(shape.H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))).to(BF)
    return moe.MoEBlock(shape, w, router, nw, residual_dtype=rt)


def _autograd(block, x, r, dout, dh, idx):
    """The block in 64 bits with the experts that the kernels chose."""
    s = block.shape
    leaf = lambda t: t.double().detach().requires_grad_(True)  # noqa: E731
    p = {k: leaf(v) for k, v in block.w.items()}
    p["w_router"], p["norm_weight"], p["dx"], p["dresidual"] = leaf(block.w_router), leaf(block.norm_weight), leaf(x), leaf(r)
    h = p["dx"] + p["dresidual"]
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + block.eps) * p["norm_weight"]
    sg = torch.sigmoid(torch.gather(n @ p["w_router"].T, 1, idx.long()))
    tw = s.scaling * (sg / sg.sum(1, keepdim=True) if s.route_norm else sg)
    ffn = lambda a, g, u, d: (torch.nn.functional.silu(a @ g.T) * (a @ u.T)) @ d.T  # noqa: E731
    rows = []
    for t in range(s.T):
        rows.append(sum(tw[t, k] * ffn(n[t], *(p[w][int(idx[t, k])] for w in ("w_gate", "w_up", "w_down")))
                        for k in range(s.K)))
    out = torch.stack(rows)
    if s.I_shared:
        out = out + ffn(n, p["ws_gate"], p["ws_up"], p["ws_down"])
    ((out * dout.double()).sum() + (h * dh.double()).sum()).backward()
    return out.detach(), h.detach(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("shape,rt", [
    (synth.MoEShape("a", T=40, H=256, E=8, K=2, I=128, I_shared=128), BF),
    (synth.MoEShape("b", T=33, H=128, E=12, K=3, I=64, I_shared=0, route_norm=False), torch.float32),
])
def test_block_against_autograd(shape, rt):
    b = _block(shape, rt)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((shape.T, shape.H), device="cuda", generator=g).to(BF)
    r = torch.randn((shape.T, shape.H), device="cuda", generator=g).to(rt)
    dout = torch.randn((shape.T, shape.H), device="cuda", generator=g).to(BF)
    dh = torch.randn((shape.T, shape.H), device="cuda", generator=g).to(rt)
    out, h = b.forward(x, r)
    grads = b.backward(dout, dh)
    want_out, want_h, want = _autograd(b, x, r, dout, dh, b.topk_idx)
    rel = lambda a, e: ((a.double() - e).norm() / e.norm()).item()  # noqa: E731
    assert rel(out, want_out) <= 2e-2 and rel(h, want_h) <= 4e-3
    for k, v in want.items():
        assert rel(grads[k], v) <= 2e-2, (k, rel(grads[k], v))
    assert b.handle.device_status() == 0


def test_gradients_in_a_cuda_graph():
    """The library's backward calls (chained launches and clusters among them) captured once and replayed."""
    shape = synth.MoEShape("g", T=96, H=256, E=8, K=2, I=128, I_shared=128)
    b = _block(shape, BF)
    x, r, dout = (torch.randn((shape.T, shape.H), device="cuda").to(BF) for _ in range(3))
    b.forward(x, r)

    def calls():
        h, w, g = b.handle, b.w, b.grads
        moe.combine_backward(h, b.cfg, dout, b.y_perm, b.topk_w, b.flat_to_perm, b.dy_perm, b.dtopk_w,
                             topk_idx=b.topk_idx, logits=b.logits, dlogits=b.dlogits)
        moe.grouped_swiglu_backward(h, b.x_perm, b.dy_perm, b.offsets, w["w_gate"], w["w_up"], w["w_down"], b.dx_perm,
                                    g["w_gate"], g["w_up"], g["w_down"], b.ws, num_groups=shape.E, H=shape.H, I=shape.I)
        moe.permute_backward(h, b.cfg, b.dx_perm, b.flat_to_perm, b.dn)
        moe.add_rmsnorm_backward(h, b.dn, b.h, b.norm_weight, b.rstd, b.dh, b.ws, dweight=g["norm_weight"])

    names = lambda: [b.dlogits, b.dx_perm, b.grads["w_gate"], b.grads["w_up"], b.grads["w_down"], b.dh,  # noqa: E731
                     b.grads["norm_weight"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [t.clone() for t in names()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        for t in names():
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(names(), want))
    assert b.handle.device_status() == 0


def test_the_example_trains_and_serves():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block_example", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.train(steps=40)
    assert losses[-1] < 0.5 * losses[0], losses[::10]
    out, _, inside = ex.serve()
    # Codes from the fp32 norm against codes from its bf16 rounding: 2^-8 / sqrt(3) into a 3-bit mantissa's
    # quantiser moves an element by at most one step now and then; the layer's output by a few 1e-2 at most.
    assert ((out.float() - inside.float()).norm() / inside.float().norm()).item() < 5e-2


def test_a_block_of_one_token():
    """Over one token nothing averages: the routing's gradient is a multiple of the difference of two experts'
    <dout, y>, whose roundings count against the sums of absolute values, not against what the difference leaves."""
    shape = synth.MoEShape("one", T=1, H=128, E=8, K=2, I=64, I_shared=64)
    b = _block(shape, BF)
    g = torch.Generator(device="cuda").manual_seed(9)
    x, r, dout = (torch.randn((1, shape.H), device="cuda", generator=g).to(BF) for _ in range(3))
    b.forward(x, r)
    grads = b.backward(dout, r)
    _, _, want = _autograd(b, x, r, dout, r, b.topk_idx)
    sg = torch.sigmoid(torch.gather(b.logits, 1, b.topk_idx.long()).double())
    w = sg / sg.sum()
    y = b.y_perm.double()[b.flat_to_perm.long()].abs()  # slot by slot
    dl = shape.scaling * w * (1 - sg) * (y @ dout.double().abs().t()).sum()  # at least the absolute sums
    size = {"w_router": dl.norm() * b.n.double().norm()}
    for k, v in want.items():
        assert (grads[k].double() - v).norm() <= 2e-2 * size.get(k, v.norm()), k
    assert b.handle.device_status() == 0
