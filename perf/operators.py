"""Cases that measure the operators around the MoE layer: the residual add + RMS norm that makes the layer's bf16 /
MXFP8 input (and its backward pass), the gradient of the token dispatch (weighted combine, routing weights, permutation),
and the gradient of the grouped SwiGLU expert products.

`own` False: plain forms in elementary 32-bit torch operations. `own` True: the library's entry points.
Shapes are the repository's workloads (hidden 4096, 192 experts, top 8, expert intermediate 1536; 64 to 8192 tokens)
and smaller generic ones.
"""
import math

import torch

own = False

EPS = 1e-5
SCALING = 2.826
MOST_ELEMENTS = 8192 * 4096  # rows * H of the largest norm case
MOST_PAIRS = 8 * 8192 * 4096  # T * K * H of the largest dispatch case
MOST_MACS = 8 * 8192 * 4096 * 1536  # rows * H * I of the largest expert case
MOST_WEIGHTS = 192 * 4096 * 1536  # groups * H * I of the largest expert case
MOST_PADDED = 1_500_000_000  # groups * T * H of a skewed expert case: its plain form pads each group to the longest


def listed():
    return [
        # A decode step's norm before an MXFP8 layer: bf16 for the router, E4M3 + E8M0 for the experts.
        {"name": "norm_decode_mx", "op": "norm", "rows": 64, "H": 4096, "res": "bf16", "mx": True},
        # The same at a prefill of 8192 tokens.
        {"name": "norm_prefill_mx", "op": "norm", "rows": 8192, "H": 4096, "res": "bf16", "mx": True},
        # A training step's forward norm on an fp32 residual stream, a ragged number of rows.
        {"name": "norm_train_f32", "op": "norm", "rows": 4093, "H": 4096, "res": "f32", "mx": False},
        # Its backward pass over a bf16 residual stream at the prefill size.
        {"name": "norm_grad", "op": "norm_grad", "rows": 8192, "H": 4096, "res": "bf16"},
        # Gradient of the weighted combine and of the routing weights: a small batch (latency), ...
        {"name": "combine_grad_small", "op": "combine_grad", "T": 61, "H": 4096, "E": 192, "K": 8, "norm": True},
        # ... and a training batch of the 192-expert layer.
        {"name": "combine_grad_large", "op": "combine_grad", "T": 8192, "H": 4096, "E": 192, "K": 8, "norm": True},
        # Gradient of the permutation with the shared expert's gradient added, ragged and small, ...
        {"name": "permute_grad_ragged", "op": "permute_grad", "T": 1021, "H": 1024, "E": 64, "K": 5, "add": False},
        # ... and at the training batch.
        {"name": "permute_grad_large", "op": "permute_grad", "T": 8192, "H": 4096, "E": 192, "K": 8, "add": True},
        # Gradient of the expert products: a few rows for each of a few small experts (latency), ...
        {"name": "experts_grad_small", "op": "experts_grad", "T": 128, "H": 1024, "I": 512, "E": 8, "K": 2, "skew": 0.0},
        # ... a skewed load with empty experts and long ones, ...
        {"name": "experts_grad_skewed", "op": "experts_grad", "T": 2048, "H": 2048, "I": 768, "E": 64, "K": 8, "skew": 2.0},
        # ... the shared expert (one group of all tokens), ...
        {"name": "experts_grad_shared", "op": "experts_grad", "T": 8192, "H": 4096, "I": 1536, "E": 1, "K": 1, "skew": 0.0},
        # ... and the 192-expert layer's training batch.
        {"name": "experts_grad_large", "op": "experts_grad", "T": 8192, "H": 4096, "I": 1536, "E": 192, "K": 8, "skew": 0.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _mult(rng, lo, hi, m):
    v = _log(rng, lo // m, hi // m) * m
    return v + m if v == 3 * 1024 else v


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "combine_grad", "permute_grad", "experts_grad"])
    if op in ("norm", "norm_grad"):
        mx = op == "norm" and rng.random() < 0.5
        H = _mult(rng, 256, 8192, 32 if mx else 8)
        rows = _log(rng, 1, min(32768, MOST_ELEMENTS // H))
        c = {"op": op, "rows": rows, "H": H, "res": rng.choice(["bf16", "f32"])}
        return dict(c, mx=mx) if op == "norm" else c
    E = _log(rng, 8, 256)
    K = rng.randint(1, 8)
    if op == "experts_grad":
        H, I = _mult(rng, 256, 4096, 64), _mult(rng, 128, 1536, 64)
        E = max(K, min(E, MOST_WEIGHTS // (H * I)))
        skew = rng.choice([0.0, 1.0, 2.0])
        T = _log(rng, 16, max(16, min(16384, MOST_MACS // (K * H * I), MOST_PADDED // (E * H) if skew else 16384)))
        return {"op": op, "T": T, "H": H, "I": I, "E": E, "K": K, "skew": skew}
    H = _mult(rng, 256, 8192, 64)
    T = _log(rng, 1, max(1, min(16384, MOST_PAIRS // (K * H))))
    c = {"op": op, "T": T, "H": H, "E": E, "K": K}
    return dict(c, norm=K > 1 and rng.random() < 0.7) if op == "combine_grad" else dict(c, add=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _out(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _routing(g, c):
    """logits [T, E], the top-K ids [T, K] and the stable order of the T*K pairs by expert: pair f sits at row
    flat_to_perm[f]."""
    logits = _normal(g, (c["T"], c["E"]), 1.0, torch.float32)
    if c.get("skew"):
        logits = logits + _normal(g, (1, c["E"]), c["skew"], torch.float32)
    idx = torch.topk(logits, c["K"], dim=1).indices.to(torch.int32)
    order = torch.argsort(idx.reshape(-1).long(), stable=True)
    f2p = torch.empty_like(order)
    f2p[order] = torch.arange(order.numel(), device=order.device)
    return logits, idx, f2p.to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    bf, f32 = torch.bfloat16, torch.float32
    s = {"c": c}
    if c["op"] in ("norm", "norm_grad"):
        rows, H, rt = c["rows"], c["H"], bf if c["res"] == "bf16" else f32
        s["w"] = (1.0 + 0.1 * _normal(g, (H,), 1.0, f32)).to(bf)
        if c["op"] == "norm":
            s["x"] = _normal(g, (rows, H), 1.0, bf)
            s["r"] = _normal(g, (rows, H), 3.0, rt)
            s["o_h"], s["o_out"], s["o_rstd"] = _out((rows, H), rt), _out((rows, H), bf), _out((rows,), f32)
            if c["mx"]:
                s["o_q"], s["o_s"] = _out((rows, H), torch.uint8), _out((rows, H // 32), torch.uint8)
        else:
            s["h"] = _normal(g, (rows, H), 3.0, rt)
            s["dout"] = _normal(g, (rows, H), 0.02, bf)
            s["dh_in"] = _normal(g, (rows, H), 0.02, rt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["o_dh"], s["o_dw"] = _out((rows, H), rt), _out((H,), f32)
        return s
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    if c["op"] == "experts_grad":
        I, R = c["I"], T * K
        if E > 1:
            _, idx, _ = _routing(g, c)
            counts = torch.bincount(idx.reshape(-1).long(), minlength=E)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            s["cap"] = int(counts.max())
        else:
            s["offsets"] = torch.tensor([0, R], dtype=torch.int32, device="cuda")
            s["cap"] = R
        s["a"] = _normal(g, (R, H), 1.0, bf)
        s["dy"] = _normal(g, (R, H), 0.01, bf)
        for n, shape in (("wg", (E, I, H)), ("wu", (E, I, H)), ("wd", (E, H, I))):
            s[n] = _normal(g, shape, 0.02, bf)
            s["o_d" + n] = _out(shape, bf)
        s["o_da"] = _out((R, H), bf)
        return s
    s["logits"], s["idx"], s["f2p"] = _routing(g, c)
    if c["op"] == "combine_grad":
        sg = torch.sigmoid(torch.gather(s["logits"], 1, s["idx"].long()))
        s["tw"] = SCALING * (sg / sg.sum(1, keepdim=True) if c["norm"] else sg)
        s["y"] = _normal(g, (T * K, H), 0.5, f32)
        s["dout"] = _normal(g, (T, H), 0.02, bf)
        s["o_dy"], s["o_dtw"], s["o_dl"] = _out((T * K, H), bf), _out((T, K), f32), _out((T, E), f32)
    else:
        s["dxp"] = _normal(g, (T * K, H), 0.02, bf)
        s["add"] = _normal(g, (T, H), 0.02, bf) if c["add"] else None
        s["o_dx"] = _out((T, H), bf)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _OWN[state["c"]["op"]](state)
    return _PLAIN[state["c"]["op"]](state)


def _norm(s):
    h = s["x"].float() + s["r"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    n = h * rstd[:, None] * s["w"].float()
    out = {"h": h.to(s["r"].dtype), "out": n.to(torch.bfloat16), "rstd": rstd}
    if s["c"]["mx"]:
        b = n.reshape(n.shape[0], -1, 32)
        amax = b.abs().amax(2)
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, torch.full_like(amax, -127, dtype=torch.int32))
        e = e.clamp(-127, 127)
        v = (b * torch.exp2(-e.float())[:, :, None]).clamp(-448.0, 448.0)
        out["q"] = v.reshape(n.shape).to(torch.float8_e4m3fn)
        out["scale"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _norm_grad(s):
    xhat = s["h"].float() * s["rstd"][:, None]
    d = s["dout"].float()
    gw = d * s["w"].float()
    dh = s["rstd"][:, None] * (gw - xhat * (gw * xhat).mean(1, keepdim=True)) + s["dh_in"].float()
    return {"dh": dh.to(s["h"].dtype), "dw": (d * xhat).sum(0)}


def _combine_grad(s):
    T, K = s["tw"].shape
    d, p = s["dout"].float(), s["f2p"].long()
    dtw = (s["y"][p].reshape(T, K, -1) * d[:, None, :]).sum(2)
    dy = torch.empty_like(s["y"], dtype=torch.bfloat16)
    dy[p] = (s["tw"][:, :, None] * d[:, None, :]).reshape(T * K, -1).to(torch.bfloat16)
    idx = s["idx"].long()
    sg = 1.0 / (1.0 + torch.exp(-torch.gather(s["logits"], 1, idx)))
    if s["c"]["norm"]:
        S = sg.sum(1, keepdim=True)
        ds = SCALING * (dtw - (dtw * sg).sum(1, keepdim=True) / S) / S
    else:
        ds = SCALING * dtw
    dl = torch.zeros_like(s["logits"])
    dl.scatter_(1, idx, ds * sg * (1.0 - sg))
    return {"dy": dy, "dtopk_w": dtw, "dlogits": dl}


def _permute_grad(s):
    T, K = s["c"]["T"], s["c"]["K"]
    dx = s["dxp"].float()[s["f2p"].long()].reshape(T, K, -1).sum(1)
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return {"dx": dx.to(torch.bfloat16)}


def _experts_grad(s):
    off, cap, R = s["offsets"].long(), s["cap"], s["a"].shape[0]
    j = torch.arange(cap, device=off.device)
    live = j[None, :] < (off[1:] - off[:-1])[:, None]  # [E, cap]
    rows = (off[:-1, None] + j[None, :]).clamp(max=R - 1)
    pad = lambda t: t.float()[rows] * live[:, :, None]  # noqa: E731
    a, dy = pad(s["a"]), pad(s["dy"])
    wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    g, u, q = a @ wg.transpose(1, 2), a @ wu.transpose(1, 2), dy @ wd
    sg = 1.0 / (1.0 + torch.exp(-g))
    h, dg, du = g * sg * u, q * u * sg * (1.0 + g * (1.0 - sg)), q * g * sg
    da = torch.empty_like(s["a"])
    da[rows[live]] = (dg @ wg + du @ wu)[live].to(torch.bfloat16)
    bf = torch.bfloat16
    return {"da": da, "dw_gate": (dg.transpose(1, 2) @ a).to(bf), "dw_up": (du.transpose(1, 2) @ a).to(bf),
            "dw_down": (dy.transpose(1, 2) @ h).to(bf)}


_PLAIN = {"norm": _norm, "norm_grad": _norm_grad, "combine_grad": _combine_grad, "permute_grad": _permute_grad,
          "experts_grad": _experts_grad}

_kept = {}


def _lib():
    """The package and the handle that a program keeps."""
    if not _kept:
        import routed_expert_ffn_04_gb300 as moe

        _kept["moe"], _kept["handle"] = moe, moe.Handle()
    return _kept["moe"], _kept["handle"]


def _cfg(moe, s):
    if "cfg" not in s:
        c = s["c"]
        s["cfg"] = moe.make_config(c["T"], c["H"], c["E"], c["K"], 64, 0, SCALING, c.get("norm", True))
    return s["cfg"]


def _ws(s, size):
    if "ws" not in s:
        s["ws"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_norm(s):
    moe, h = _lib()
    out = {"h": s["o_h"], "out": s["o_out"], "rstd": s["o_rstd"]}
    moe.add_rmsnorm(h, s["x"], s["w"], EPS, residual=s["r"], h_out=s["o_h"], out=s["o_out"], q=s.get("o_q"),
                    q_scale=s.get("o_s"), rstd=s["o_rstd"])
    if s["c"]["mx"]:
        out["q"], out["scale"] = s["o_q"].view(torch.float8_e4m3fn), s["o_s"].view(torch.float8_e8m0fnu)
    return out


def _own_norm_grad(s):
    moe, h = _lib()
    ws = _ws(s, lambda: moe.add_rmsnorm_backward_workspace_size(s["c"]["rows"], s["c"]["H"]))
    moe.add_rmsnorm_backward(h, s["dout"], s["h"], s["w"], s["rstd"], s["o_dh"], ws, dh_in=s["dh_in"], dweight=s["o_dw"])
    return {"dh": s["o_dh"], "dw": s["o_dw"]}


def _own_combine_grad(s):
    moe, h = _lib()
    moe.combine_backward(h, _cfg(moe, s), s["dout"], s["y"], s["tw"], s["f2p"], s["o_dy"], s["o_dtw"],
                         topk_idx=s["idx"], logits=s["logits"], dlogits=s["o_dl"])
    return {"dy": s["o_dy"], "dtopk_w": s["o_dtw"], "dlogits": s["o_dl"]}


def _own_permute_grad(s):
    moe, h = _lib()
    moe.permute_backward(h, _cfg(moe, s), s["dxp"], s["f2p"], s["o_dx"], dx_add=s["add"])
    return {"dx": s["o_dx"]}


def _own_experts_grad(s):
    moe, h = _lib()
    c = s["c"]
    ws = _ws(s, lambda: moe.grouped_gemm_backward_workspace_size(c["T"] * c["K"], c["H"], c["I"], num_groups=c["E"]))
    moe.grouped_swiglu_backward(h, s["a"], s["dy"], s["offsets"], s["wg"], s["wu"], s["wd"], s["o_da"], s["o_dwg"],
                                s["o_dwu"], s["o_dwd"], ws, num_groups=c["E"], H=c["H"], I=c["I"])
    return {"da": s["o_da"], "dw_gate": s["o_dwg"], "dw_up": s["o_dwu"], "dw_down": s["o_dwd"]}


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "combine_grad": _own_combine_grad,
        "permute_grad": _own_permute_grad, "experts_grad": _own_experts_grad}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "norm":
        r = 2 if c["res"] == "bf16" else 4
        n = c["rows"] * c["H"]
        return {"bytes": n * (2 + 2 * r + 2 + (33 / 32 if c["mx"] else 0)) + 4 * c["rows"] + 2 * c["H"], "flops": 6 * n}
    if c["op"] == "norm_grad":
        r = 2 if c["res"] == "bf16" else 4
        n = c["rows"] * c["H"]
        return {"bytes": n * (2 + 3 * r) + 4 * c["rows"] + 6 * c["H"], "flops": 12 * n}
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    if c["op"] == "combine_grad":
        return {"bytes": T * K * H * 6 + T * H * 2 + T * K * 16 + T * E * 4 + T * K * 4, "flops": 3 * T * K * H}
    if c["op"] == "permute_grad":
        return {"bytes": T * K * H * 2 + T * H * (4 if c["add"] else 2) + T * K * 4, "flops": T * K * H}
    R, I = T * K, c["I"]
    return {"bytes": 6 * R * H + 12 * E * H * I + 4 * (E + 1), "flops": 16 * R * H * I}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: t.to(torch.float64)  # noqa: E731
    c, op = case, case["op"]
    if op == "norm":
        v = d(s["x"]).add_(d(s["r"]))
        ms = torch.linalg.vector_norm(v, dim=1).square() / c["H"]
        rstd = (ms + EPS).pow(-0.5)
        n = torch.einsum("rh,r,h->rh", v, rstd, d(s["w"]))
        q = scale = None
        if c["mx"]:
            blocks = n.unflatten(1, (-1, 32))
            top = blocks.abs().max(dim=2).values
            k = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 8, torch.full_like(top, -127.0))
            k = k.clamp(-127, 127)
            q = _e4m3(torch.ldexp(blocks, -k[:, :, None])).flatten(1)
            scale = torch.exp2(k)
        out = {"h": v, "out": n, "rstd": rstd}
        return dict(out, q=q, scale=scale) if c["mx"] else out
    if op == "norm_grad":
        z = torch.einsum("rh,r->rh", d(s["h"]), d(s["rstd"]))
        do, w = d(s["dout"]), d(s["w"])
        m = torch.einsum("rh,h,rh->r", do, w, z) / c["H"]
        dh = d(s["dh_in"]) + torch.einsum("r,rh->rh", d(s["rstd"]), do * w - torch.einsum("rh,r->rh", z, m))
        return {"dh": dh, "dw": torch.einsum("rh,rh->h", do, z)}
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    if op == "combine_grad":
        f = s["f2p"].long().view(T, K)
        do, tw, l = d(s["dout"]), d(s["tw"]), d(s["logits"])
        dy = torch.empty((T * K, H), dtype=torch.float64, device="cuda")
        dtw = torch.empty((T, K), dtype=torch.float64, device="cuda")
        for k in range(K):
            dy.index_copy_(0, f[:, k], tw[:, k, None] * do)
            dtw[:, k] = torch.einsum("th,th->t", d(s["y"].index_select(0, f[:, k])), do)
        pick = torch.zeros((T, E), dtype=torch.float64, device="cuda")
        pick.scatter_(1, s["idx"].long(), 1.0)
        full = torch.zeros_like(pick).scatter_(1, s["idx"].long(), dtw)
        sg = torch.special.expit(l)
        grad = full * SCALING
        if c["norm"]:  # d (s_k / S) / d s_j = (delta_kj - s_k / S) / S
            S = torch.einsum("te,te->t", pick, sg)[:, None]
            grad = pick * (grad - torch.einsum("te,te->t", grad, sg)[:, None] / S) / S
        return {"dy": dy, "dtopk_w": dtw, "dlogits": grad * sg * torch.special.expit(-l)}
    if op == "permute_grad":
        dx = d(s["add"]) if s["add"] is not None else torch.zeros((T, H), dtype=torch.float64, device="cuda")
        f = s["f2p"].long().view(T, K)
        for k in range(K):
            dx = dx + d(s["dxp"].index_select(0, f[:, k]))
        return {"dx": dx}
    R, I = T * K, c["I"]
    out = {n: torch.zeros(sh, dtype=torch.float64, device="cuda") for n, sh in
           (("da", (R, H)), ("dw_gate", (E, I, H)), ("dw_up", (E, I, H)), ("dw_down", (E, H, I)))}
    off = s["offsets"].tolist()
    for e in range(E):
        b, n = off[e], off[e + 1]
        if b == n:
            continue
        x, gy, wg, wu, wd = (d(t) for t in (s["a"][b:n], s["dy"][b:n], s["wg"][e], s["wu"][e], s["wd"][e]))
        gate, up, gh = torch.mm(x, wg.t()), torch.mm(x, wu.t()), torch.mm(gy, wd)
        sg = torch.special.expit(gate)
        act = gate * sg
        out["dw_down"][e] = torch.mm(gy.t(), act * up)
        ggate, gup = gh * up * (sg + act * (1 - sg)), gh * act
        out["dw_gate"][e], out["dw_up"][e] = torch.mm(ggate.t(), x), torch.mm(gup.t(), x)
        out["da"][b:n] = torch.addmm(torch.mm(ggate, wg), gup, wu)
    return out


def _e4m3(v):
    """Nearest E4M3 number (ties to even), saturating at 448."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)
