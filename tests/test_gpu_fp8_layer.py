"""The layer with E4M3 operands and fp32 scales per block of 128 ("fp8"), its pieces run together, and the block with
its balance loss.

Tolerance of the layer against its definition in 64 bits: both quantise x and the weights alike; h differs where a
value lies within fp32 rounding of a border between codes (about 1e-5 of them, each by at most 2^-3), which is below
1e-3 of the output's norm; the output is rounded to bf16 once: 2^-8 of each value at most."""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe
import synth
from test_gpu_balance import share_tol
from test_gpu_fp8 import quantize64, rows64, squares64

pytestmark = pytest.mark.gpu

F64 = torch.float64
SHAPES = [synth.WORKLOADS["tiny"].with_(dtype="fp8"), synth.MoEShape("fr", T=45, H=384, E=13, K=3, I=256, I_shared=128, dtype="fp8"),
          synth.MoEShape("fn", T=1, H=128, E=5, K=2, I=128, I_shared=0, dtype="fp8"),
          synth.MoEShape("fs", T=700, H=640, E=6, K=2, I=384, I_shared=256, dtype="fp8", skew=True)]


def problem(shape, seed=0):
    x, logits = synth.make_activations(shape, device="cuda", seed=seed)
    return x, logits, synth.make_weights(shape, device="cuda", seed=seed)


def mlp64(q, s, wg, wu, wd):
    """SwiGLU of the values that codes stand for, h quantised by the rule on its fp32 rounding."""
    x = rows64(q, s)
    gate, up = x @ wg.t(), x @ wu.t()
    hq, hs = quantize64((gate * torch.sigmoid(gate) * up).float(), 1, 128)
    return rows64(hq, hs) @ wd.t()


def layer64(shape, x, logits, w):
    val = {k: [squares64(*quantize64(m, 128, 128)) for m in (v if v.dim() == 3 else v[None])] for k, v in w.items()}
    q, s = quantize64(x, 1, 128)
    sg, idx = torch.sigmoid(logits.to(F64)), torch.topk(logits, shape.K, dim=1).indices
    tw = torch.gather(sg, 1, idx)
    tw = shape.scaling * (tw / tw.sum(1, keepdim=True) if shape.route_norm else tw)
    out = torch.zeros((shape.T, shape.H), dtype=F64, device="cuda")
    for e in range(shape.E):
        t, k = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            y = mlp64(q[t], s[t], val["w_gate"][e], val["w_up"][e], val["w_down"][e])
            out.index_add_(0, t, tw[t, k][:, None] * y)
    if shape.I_shared:
        out += mlp64(q, s, val["ws_gate"][0], val["ws_up"][0], val["ws_down"][0])
    return out


@pytest.mark.parametrize("side", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s.name)
def test_layer(shape, side):
    x, logits, w = problem(shape)
    layer = moe.MoELayer(shape, w, device=0, side_stream=side)
    out = layer(x, logits)
    torch.cuda.synchronize()
    assert layer.handle.device_status() == 0
    ref = layer64(shape, x, logits, w)
    err = out.to(F64) - ref
    assert float(err.norm() / ref.norm()) <= 2.0 ** -8 + 1e-3


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s.name)
def test_layer_is_its_pieces(shape):
    """The same bits from route, quantize_fp8, permute, grouped_swiglu_gemm (and its two halves) and combine."""
    x, logits, w = problem(shape, 1)
    layer = moe.MoELayer(shape, w, device=0)
    h, cfg, wq, T, H, E, K, I = layer.handle, layer.cfg, layer.weights_t, shape.T, shape.H, shape.E, shape.K, shape.I
    out = layer(x, logits)
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    i32, u8, bf = torch.int32, torch.uint8, torch.bfloat16
    idx, tw, q, s = e(T, K, dt=i32), e(T, K), e(T, H, dt=u8), e(T, H // 128)
    moe.route(h, cfg, logits, idx, tw)
    moe.quantize_fp8(h, x, q, s)
    counts, off, src, f2p = e(E, dt=i32), e(E + 1, dt=i32), e(T * K, dt=i32), e(T * K, dt=i32)
    xp, sp = e(T * K, H, dt=u8), e(T * K, H // 128)
    ws = e(max(moe.permute_workspace_size(cfg), moe.grouped_gemm_workspace_size(T * max(K, 1), H, max(I, shape.I_shared), moe.MOE_FP8_BLOCK128, E)), dt=u8)
    moe.permute(h, cfg, q, idx, counts, off, src, f2p, xp, ws, x_scale=s.view(u8), x_perm_scale=sp.view(u8))
    y, ys = e(T * K, H), None
    moe.grouped_swiglu_gemm(h, xp, off, wq["w_gate"], wq["w_up"], wq["w_down"], y, ws, num_groups=E, H=H, I=I,
                            dtype=moe.MOE_FP8_BLOCK128, a_scale=sp, s_gate=wq["s_gate"], s_up=wq["s_up"], s_down=wq["s_down"])
    if shape.I_shared:
        ys = e(T, H)
        moe.grouped_swiglu_gemm(h, q, None, wq["ws_gate"], wq["ws_up"], wq["ws_down"], ys, ws, num_groups=1, H=H, I=shape.I_shared,
                                dtype=moe.MOE_FP8_BLOCK128, a_scale=s, s_gate=wq["ss_gate"], s_up=wq["ss_up"], s_down=wq["ss_down"])
    out2 = e(T, H, dt=bf)
    moe.combine(h, cfg, y, tw, f2p, ys, out2)
    assert torch.equal(out, out2)
    hq, hs, y2 = e(T * K, I, dt=u8), e(T * K, I // 128), e(T * K, H)
    moe.grouped_gate_up_fp8(h, xp, sp, off, wq["w_gate"], wq["s_gate"], wq["w_up"], wq["s_up"], hq, hs, num_groups=E, H=H, I=I)
    moe.grouped_gemm_fp8(h, hq, hs, off, wq["w_down"], wq["s_down"], y2, num_groups=E, N=H, K=I)
    assert torch.equal(y, y2)
    # x already quantised
    assert torch.equal(layer(q, logits, x_scale=s), out)
    # a permutation without a workspace moves the same bytes
    xp2, sp2 = torch.empty_like(xp), torch.empty_like(sp)
    moe.permute_static_scratch(h, cfg, q, idx, counts, off, src, f2p, xp2, x_scale=s.view(u8), x_perm_scale=sp2.view(u8))
    assert torch.equal(xp, xp2) and torch.equal(sp, sp2)


def test_shared_expert_on_few_sms():
    """The shared expert's products stay on the SMs that an option gives them: its reduction is not shared out then."""
    shape = synth.MoEShape("fd", T=9, H=4096, E=3, K=1, I=128, I_shared=256, dtype="fp8")
    x, logits, w = problem(shape, 2)
    layer = moe.MoELayer(shape, w, device=0)
    out = layer(x, logits)
    layer.handle.set_option(moe.MOE_OPT_SHARED_SMS, 8)
    few = layer(x, logits)
    ref = layer64(shape, x, logits, w)
    for o in (out, few):
        assert float((o.to(F64) - ref).norm() / ref.norm()) <= 2.0 ** -8 + 1e-3
    assert layer.handle.device_status() == 0


def test_layer_in_a_graph_host_and_gated():
    shape = SHAPES[1]
    x, logits, w = problem(shape, 2)
    layer = moe.MoELayer(shape, w, device=0)
    out = layer(x, logits).clone()
    again = torch.empty_like(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, logits, out=again)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    host = torch.empty(out.shape, dtype=out.dtype, pin_memory=True)
    moe.layer_forward_host(layer.handle, layer.cfg, layer.weights, x.cpu().pin_memory(), logits.cpu().pin_memory(), host,
                           layer.ws, side=layer.side)
    assert torch.equal(host, out.cpu())
    router = synth.make_router(shape, device="cuda", seed=2)
    gated = torch.empty_like(out)
    moe.layer_forward_gated(layer.handle, layer.cfg, layer.weights, router, x, gated, layer.ws, side=layer.side)
    lg = torch.empty((shape.T, shape.E), device="cuda")
    idx, tw = torch.empty((shape.T, shape.K), dtype=torch.int32, device="cuda"), torch.empty((shape.T, shape.K), device="cuda")
    moe.gate_route(layer.handle, layer.cfg, x, router, idx, tw, logits_out=lg)
    assert torch.equal(gated, layer(x, lg)) and layer.handle.device_status() == 0


def test_refusals():
    c = moe.make_config(8, 192, 4, 2, 128, 0, 1.0, dtype=moe.MOE_FP8_BLOCK128)
    with pytest.raises(moe.MoEError):  # H in whole blocks of 128
        moe.workspace_size(c)
    with pytest.raises(moe.MoEError) as e:  # the SwiGLU experts' gradient is bf16's
        moe.grouped_gemm_backward_workspace_size(8, 256, 128, moe.MOE_FP8_BLOCK128)
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED


# ---------------------------------------------------------------- the block's balance loss
def block(shape, coef, seed=0):
    w = synth.make_weights(shape, device="cuda", seed=seed, std=0.05)
    router = synth.make_router(shape, device="cuda", seed=seed, std=0.05)
    return moe.MoEBlock(shape, w, router, torch.ones(shape.H, dtype=torch.bfloat16, device="cuda"), balance_coef=coef)


def test_block_balance():
    """The loss and counts of the block's own logits, and the gradient's way to the router and the input."""
    shape = synth.WORKLOADS["tiny"].with_(T=200, H=256, E=16, K=4, I=128, I_shared=128)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dout = (torch.randn((shape.T, shape.H), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    plain, bal = block(shape, 0.0), block(shape, 0.5)
    out0, _ = plain.forward(x)
    out1, _ = bal.forward(x)
    assert torch.equal(out0, out1) and torch.equal(plain.logits, bal.logits)
    p = torch.sigmoid(bal.logits.to(F64))
    p = p / p.sum(1, keepdim=True)
    load = torch.bincount(bal.topk_idx.reshape(-1).long(), minlength=shape.E)
    assert torch.equal(bal.load[0].long(), load)
    f = load.to(F64) * shape.E / (shape.K * shape.T)
    want = 0.5 * (f * p.mean(0)).sum()
    assert abs(float(bal.balance) - float(want)) <= 1e-5 * float(want)
    plain.backward(dout)
    two = torch.full((1,), 2.0, device="cuda")
    for scale, kw in ((1.0, {}), (2.0, dict(dbalance=two))):
        bal.backward(dout, **kw)
        d = scale * 0.5 / shape.T * (f - (p * f).sum(1, keepdim=True)) * p * torch.sigmoid(-bal.logits.to(F64))
        got = bal.dlogits.to(F64) - plain.dlogits.to(F64)
        # f and its mean are subtracted in fp32, off by share_tol of themselves (test_gpu_balance); then the sum's rounding
        size = scale * 0.5 / shape.T * (f + (p * f).sum(1, keepdim=True)) * p
        tol = size * (2 * share_tol(shape.E) + 2.0 ** -20) + 2.0 ** -22 * (plain.dlogits.abs() + d.abs())
        assert ((got - d).abs() <= tol).all()
    assert not torch.equal(plain.grads["w_router"], bal.grads["w_router"])
    assert torch.equal(plain.grads["w_gate"], bal.grads["w_gate"])
