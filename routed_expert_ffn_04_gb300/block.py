"""The MoE block around the layer, for training (bf16): residual add + RMS norm, gating, routed and shared experts,
forward and backward, on the library's kernels. The gating projection's two gradient products are plain matrix
products (torch)."""
from __future__ import annotations

import torch

import routed_expert_ffn_04_gb300 as moe


class MoEBlock:
    """h = x + residual; n = RMSNorm(h) * norm_weight; out = MoE(n), with the buffers for one shape.

    weights: w_gate, w_up [E, I, H], w_down [E, H, I], and with I_shared > 0 ws_gate, ws_up [I_shared, H], ws_down
    [H, I_shared]; w_router [E, H]; norm_weight [H]; all bf16 on the block's device. forward() keeps what backward()
    needs until the next forward(); the tensors they return are the block's own buffers."""

    def __init__(self, shape, weights: dict, w_router, norm_weight, eps: float = 1e-5, residual_dtype=torch.bfloat16):
        if shape.dtype != "bf16":
            raise ValueError("MoEBlock trains bf16 layers")
        self.shape, self.w, self.w_router, self.norm_weight, self.eps = shape, weights, w_router, norm_weight, eps
        self.dev = w_router.device
        self.handle = moe.Handle(self.dev.index)
        s = shape
        self.cfg = moe.make_config(s.T, s.H, s.E, s.K, s.I, s.I_shared, s.scaling, s.route_norm)
        bf, f32, i32, rt = torch.bfloat16, torch.float32, torch.int32, residual_dtype
        new = lambda *sz, dt=bf: torch.empty(sz, dtype=dt, device=self.dev)  # noqa: E731
        T, H, E, K, TK = s.T, s.H, s.E, s.K, s.T * s.K
        self.h, self.n, self.rstd, self.out = new(T, H, dt=rt), new(T, H), new(T, dt=f32), new(T, H)
        self.logits, self.topk_idx, self.topk_w = new(T, E, dt=f32), new(T, K, dt=i32), new(T, K, dt=f32)
        self.counts, self.offsets = new(E, dt=i32), new(E + 1, dt=i32)
        self.perm_src, self.flat_to_perm = new(TK, dt=i32), new(TK, dt=i32)
        self.x_perm, self.y_perm = new(TK, H), new(TK, H, dt=f32)
        self.shared = new(T, H, dt=f32) if s.I_shared else None
        self.dy_perm, self.dx_perm, self.dn = new(TK, H), new(TK, H), new(T, H)
        self.dtopk_w, self.dlogits = new(T, K, dt=f32), new(T, E, dt=f32)
        self.dh, self.dx = new(T, H, dt=rt), new(T, H)
        self.grads = {k: torch.empty_like(v) for k, v in weights.items()}
        self.grads["norm_weight"] = new(H, dt=f32)
        self.dn_shared = new(T, H) if s.I_shared else None
        sizes = [moe.permute_workspace_size(self.cfg), moe.grouped_gemm_workspace_size(TK, H, s.I, num_groups=E),
                 moe.grouped_gemm_backward_workspace_size(TK, H, s.I, num_groups=E),
                 moe.add_rmsnorm_backward_workspace_size(T, H)]
        if s.I_shared:
            sizes += [moe.grouped_gemm_workspace_size(T, H, s.I_shared),
                      moe.grouped_gemm_backward_workspace_size(T, H, s.I_shared)]
        self.ws = torch.empty(max(sizes), dtype=torch.uint8, device=self.dev)  # one stream: the calls take turns

    def forward(self, x, residual=None, stream=None):
        """x [T, H] bf16, residual [T, H] or None -> (out [T, H] bf16, h [T, H], the residual stream's new value)."""
        s, h, cfg, w = self.shape, self.handle, self.cfg, self.w
        moe.add_rmsnorm(h, x, self.norm_weight, self.eps, residual=residual, h_out=self.h, out=self.n, rstd=self.rstd,
                        stream=stream)
        moe.gate_route(h, cfg, self.n, self.w_router, self.topk_idx, self.topk_w, logits_out=self.logits, stream=stream)
        moe.permute(h, cfg, self.n, self.topk_idx, self.counts, self.offsets, self.perm_src, self.flat_to_perm,
                    self.x_perm, self.ws, stream=stream)
        moe.grouped_swiglu_gemm(h, self.x_perm, self.offsets, w["w_gate"], w["w_up"], w["w_down"], self.y_perm, self.ws,
                                num_groups=s.E, H=s.H, I=s.I, stream=stream)
        if s.I_shared:
            moe.grouped_swiglu_gemm(h, self.n, None, w["ws_gate"], w["ws_up"], w["ws_down"], self.shared, self.ws,
                                    num_groups=1, H=s.H, I=s.I_shared, stream=stream)
        moe.combine(h, cfg, self.y_perm, self.topk_w, self.flat_to_perm, self.shared, self.out, stream=stream)
        return self.out, self.h

    def backward(self, dout, dh=None, stream=None):
        """dout [T, H] bf16 (gradient of out), dh (gradient of h on its own path, the stream's type, or None) ->
        gradients by name: dx and dresidual, norm_weight and w_router (fp32), and the expert weights (bf16)."""
        s, h, cfg, w, g = self.shape, self.handle, self.cfg, self.w, self.grads
        moe.combine_backward(h, cfg, dout, self.y_perm, self.topk_w, self.flat_to_perm, self.dy_perm, self.dtopk_w,
                             topk_idx=self.topk_idx, logits=self.logits, dlogits=self.dlogits, stream=stream)
        moe.grouped_swiglu_backward(h, self.x_perm, self.dy_perm, self.offsets, w["w_gate"], w["w_up"], w["w_down"],
                                    self.dx_perm, g["w_gate"], g["w_up"], g["w_down"], self.ws, num_groups=s.E, H=s.H,
                                    I=s.I, stream=stream)
        if s.I_shared:
            moe.grouped_swiglu_backward(h, self.n, dout, None, w["ws_gate"], w["ws_up"], w["ws_down"], self.dn_shared,
                                        g["ws_gate"], g["ws_up"], g["ws_down"], self.ws, num_groups=1, H=s.H,
                                        I=s.I_shared, stream=stream)
        moe.permute_backward(h, cfg, self.dx_perm, self.flat_to_perm, self.dn, dx_add=self.dn_shared, stream=stream)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(self.dev):
            g["w_router"] = self.dlogits.t() @ self.n.float()
            self.dn += self.dlogits @ self.w_router.float()
        f32 = self.h.dtype == torch.float32
        moe.add_rmsnorm_backward(h, self.dn, self.h, self.norm_weight, self.rstd, self.dh, self.ws, dh_in=dh,
                                 dx=self.dx if f32 else None, dweight=g["norm_weight"], stream=stream)
        return dict(g, dx=self.dx if f32 else self.dh, dresidual=self.dh)
