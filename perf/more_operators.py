"""Cases that measure the router's balance loss (with per-expert counts and its gradient) and the experts' products in
8-bit floating point with one fp32 scale per block of 128: the quantisers, the grouped product (forward, and with the
weights transposed as the gradient of its input needs them), the gate/up product with SwiGLU whose result leaves
quantised, and the weights' gradient.

`own` False: plain forms in elementary 32-bit torch operations. `own` True: the library's entry points.
Shapes are the repository's workloads (hidden 4096, 192 or 256 experts, top 8, expert intermediate 1536; 64 to 8192
tokens) and smaller generic ones.
"""
import math

import torch

own = False

COEF = 0.01
BLOCK = 128  # elements that share a scale along a row, rows that share one along a column
E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -126
MOST_LOGITS = 65536 * 256  # T * E of the largest balance case
MOST_VALUES = 8192 * 4096  # values of the largest quantiser case
MOST_MACS = 8 * 8192 * 4096 * 1536  # rows * N * K of the largest product
MOST_WEIGHTS = 192 * 4096 * 1536  # groups * N * K of the largest product
MOST_PADDED = 600_000_000  # groups * T * columns of an uneven case: the plain forms pad each group to the longest


def listed():
    return [
        # The balance loss of a small training batch (latency), sigmoid scores as the router's.
        {"name": "balance_small", "op": "balance", "grad": False, "T": 1021, "E": 64, "K": 5, "score": "sigmoid",
         "B": 1, "pad": 0, "add": False},
        # The same per sequence: ragged sequences packed in one batch with padding behind them, softmax scores, ...
        {"name": "balance_sequences", "op": "balance", "grad": False, "T": 65536, "E": 256, "K": 8, "score": "softmax",
         "B": 29, "pad": 501, "add": False},
        # ... and the gradient that it adds to the routing weights' at the 192-expert layer's training batch.
        {"name": "balance_grad", "op": "balance", "grad": True, "T": 8192, "E": 192, "K": 8, "score": "sigmoid",
         "B": 1, "pad": 0, "add": True},
        # A prefill's activations to 8 bits, one scale per 128 values of a row.
        {"name": "quantize_rows", "op": "quantize", "form": "rows", "rows": 8192, "C": 4096, "x": "bf16"},
        # A training batch's permuted rows to 8 bits along the tokens, for the weights' gradient: uneven experts.
        {"name": "quantize_columns", "op": "quantize", "form": "columns", "T": 2048, "C": 2048, "E": 64, "K": 8,
         "skew": 2.0, "x": "bf16"},
        # A few tokens through one dense projection (latency).
        {"name": "product_few", "op": "product", "T": 7, "N": 1536, "K": 4096, "E": 1, "top": 1, "skew": 0.0,
         "transposed": False, "out": "bf16"},
        # The gradient of an input: uneven experts, weights read along their other axis.
        {"name": "product_transposed", "op": "product", "T": 2048, "N": 2048, "K": 768, "E": 64, "top": 8, "skew": 2.0,
         "transposed": True, "out": "bf16"},
        # The down projection of the 192-expert layer's prefill, fp32 rows for the combine.
        {"name": "product_prefill", "op": "product", "T": 8192, "N": 4096, "K": 1536, "E": 192, "top": 8, "skew": 0.0,
         "transposed": False, "out": "f32"},
        # Gate and up of a decode step of 64 tokens: the weights' bytes, ...
        {"name": "gate_up_decode", "op": "gate_up", "T": 64, "H": 4096, "I": 1536, "E": 192, "top": 8, "skew": 0.0},
        # ... and of the prefill.
        {"name": "gate_up_prefill", "op": "gate_up", "T": 8192, "H": 4096, "I": 1536, "E": 192, "top": 8, "skew": 0.0},
        # The weights' gradient of a few small experts (latency), ...
        {"name": "weight_grad_small", "op": "weight_grad", "T": 128, "N": 512, "K": 1024, "E": 8, "top": 2,
         "skew": 0.0},
        # ... and of one of the 192-expert layer's matrices over the training batch.
        {"name": "weight_grad_large", "op": "weight_grad", "T": 8192, "N": 1536, "K": 4096, "E": 192, "top": 8,
         "skew": 0.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _mult(rng, lo, hi, m):
    return _log(rng, lo // m, hi // m) * m


def draw(rng):
    op = rng.choice(["balance", "balance", "quantize", "product", "product", "gate_up", "weight_grad"])
    if op == "balance":
        E = _log(rng, 2, 512)
        T = _log(rng, 1, MOST_LOGITS // E // 2 if E < 64 else MOST_LOGITS // E)
        grad = rng.random() < 0.5
        B = 1 if rng.random() < 0.4 else rng.randint(2, 100)
        return {"op": op, "grad": grad, "T": T, "E": E, "K": rng.randint(1, min(E, 8)),
                "score": rng.choice(["sigmoid", "softmax"]), "B": B, "pad": rng.randint(0, T // 4) if B > 1 else 0,
                "add": grad and rng.random() < 0.5}
    if op == "quantize":
        form, x = rng.choice(["rows", "squares", "columns"]), rng.choice(["bf16", "f32"])
        if form == "columns":
            E, K = _log(rng, 1, 256), rng.randint(1, 8)
            K = min(E, K)
            C = _mult(rng, 128, 4096, 16)
            T = _log(rng, 1, max(1, min(16384, MOST_VALUES // (C * K))))
            return {"op": op, "form": form, "T": T, "C": C, "E": E, "K": K, "skew": rng.choice([0.0, 2.0]), "x": x}
        C = _mult(rng, 128, 8192, 16)
        return {"op": op, "form": form, "rows": _log(rng, 1, min(65536, MOST_VALUES // C)), "C": C, "x": x}
    E = _log(rng, 1, 256)
    top = min(E, rng.randint(1, 8))
    a, b = _mult(rng, 128, 4096, 16), _mult(rng, 128, 4096, 16)
    E = max(top, min(E, MOST_WEIGHTS // (2 * a * b)))
    skew = rng.choice([0.0, 1.0, 2.0]) if E > 1 else 0.0
    most = MOST_MACS // (2 * top * a * b)
    T = _log(rng, 1, max(1, min(16384, most, MOST_PADDED // (E * max(a, b)) if skew else 16384)))
    c = {"op": op, "T": T, "E": E, "top": top, "skew": skew}
    if op == "gate_up":
        return dict(c, H=a, I=b)
    c = dict(c, N=a, K=b)
    return c if op == "weight_grad" else dict(c, transposed=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------- inputs
def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _out(shape, dtype):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _codes(g, shape):
    """E4M3 codes as the quantisers leave them: normal values whose block's largest sits near 448."""
    return _normal(g, shape, 130.0, torch.bfloat16).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(g, shape, std):
    """Scales of blocks of values of standard deviation `std`."""
    return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(0.8, 1.25, generator=g).mul_(std / 130.0)


def _blocks(n):
    return -(-n // BLOCK)


def _routing(g, T, E, K, skew):
    """The top-K ids [T, K] of normal logits, with a bias per expert of standard deviation `skew`, and the logits."""
    logits = _normal(g, (T, E), 1.0, torch.float32)
    if skew:
        logits = logits + _normal(g, (1, E), skew, torch.float32)
    return logits, torch.topk(logits, K, dim=1).indices.to(torch.int32)


def _groups(g, s, c):
    """offsets [E + 1] of the rows of each expert, and the longest group."""
    E, K = c["E"], c["top"] if "top" in c else c["K"]
    if E > 1:
        _, idx = _routing(g, c["T"], E, K, c["skew"])
        counts = torch.bincount(idx.reshape(-1).long(), minlength=E)
    else:
        counts = torch.tensor([c["T"]], device="cuda")
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["cap"] = int(counts.max())
    s["starts"] = torch.cat([counts.new_zeros(1), ((counts + BLOCK - 1) // BLOCK * BLOCK).cumsum(0)])
    return c["T"] * K


def _padded(rows, E):
    """Rows that hold any `rows` rows in E groups, each padded to a multiple of 128."""
    return (rows // BLOCK + E) * BLOCK


def _sequences(g, c):
    """Ends of B sequences of random lengths (some may be empty) in T - pad tokens."""
    cuts = torch.randint(0, c["T"] - c["pad"] + 1, (c["B"] - 1,), generator=g, device="cuda").sort().values
    ends = torch.tensor([0, c["T"] - c["pad"]], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    s = {"c": c}
    if c["op"] == "balance":
        T, E, K, B = c["T"], c["E"], c["K"], c["B"]
        s["logits"], s["idx"] = _routing(g, T, E, K, 0.5)
        s["seq"] = _sequences(g, c) if B > 1 else None
        if c["grad"]:
            s["counts"] = _counts(s)
            s["dloss"] = torch.empty((B,), dtype=f32, device="cuda").uniform_(0.5, 1.5, generator=g)
            s["add"] = _normal(g, (T, E), COEF / (T * E), f32) if c["add"] else None
            s["o_dl"] = _out((T, E), f32)
        else:
            s["o_counts"], s["o_prob"], s["o_loss"] = _out((B, E), torch.int32), _out((B, E), f32), _out((B,), f32)
        return s
    if c["op"] == "quantize":
        xt, C = bf if c["x"] == "bf16" else f32, c["C"]
        if c["form"] == "columns":
            rows = _groups(g, s, c)
            s["o_q"] = _out((_padded(rows, c["E"]), C), u8)
            s["o_s"] = _out((_padded(rows, c["E"]) // BLOCK, C), f32)
        else:
            rows = c["rows"]
            s["o_q"] = _out((rows, C), u8)
            s["o_s"] = _out((rows if c["form"] == "rows" else _blocks(rows), _blocks(C)), f32)
        s["x"] = _normal(g, (rows, C), 1.0, xt)
        return s
    E, rows = c["E"], _groups(g, s, c)
    if c["op"] == "product":
        N, K = c["N"], c["K"]
        a, b = (K, N) if c["transposed"] else (N, K)
        s["w"], s["ws"] = _codes(g, (E, a, b)), _scales(g, (E, _blocks(a), _blocks(b)), 0.02)
        s["a"], s["as"] = _codes(g, (rows, K)), _scales(g, (rows, _blocks(K)), 1.0)
        s["o"] = _out((rows, N), bf if c["out"] == "bf16" else f32)
    elif c["op"] == "gate_up":
        H, I = c["H"], c["I"]
        for n in ("g", "u"):
            s["w" + n], s["s" + n] = _codes(g, (E, I, H)), _scales(g, (E, _blocks(I), _blocks(H)), 0.02)
        s["a"], s["as"] = _codes(g, (rows, H)), _scales(g, (rows, _blocks(H)), 1.0)
        s["o_q"], s["o_s"] = _out((rows, I), u8), _out((rows, _blocks(I)), f32)
    else:
        N, K, P = c["N"], c["K"], _padded(rows, E)
        live = _live_rows(s, P)
        for n, C, std in (("dy", N, 0.01), ("a", K, 1.0)):
            s[n] = _codes(g, (P, C)) * live[:, None]
            s[n + "s"] = _scales(g, (P // BLOCK, C), std)
        s["o"] = _out((E, N, K), bf)
    return s


def _live_rows(s, P):
    """1 for the rows of [0, P) that hold a group's row, 0 for those that pad it."""
    group, at = _padded_rows(s, P)
    return (at < (s["offsets"][1:] - s["offsets"][:-1]).long()[group]).to(torch.uint8)


def _padded_rows(s, P):
    """Group and place within it of each padded row (those after the last group: a place past any row)."""
    r = torch.arange(P, device="cuda")
    group = (torch.searchsorted(s["starts"], r, right=True) - 1).clamp(0, s["starts"].numel() - 2)
    at = torch.where(r < s["starts"][-1], r - s["starts"][group], torch.full_like(r, 1 << 40))
    return group, at


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _OWN[state["c"]["op"]](state)
    return _PLAIN[state["c"]["op"]](state)


def _seq_of(s):
    """The sequence of each token, and the tokens of each sequence; a token behind the last one is of sequence B."""
    T, B = s["logits"].shape[0], s["c"]["B"]
    if s["seq"] is None:
        return torch.zeros(T, dtype=torch.long, device="cuda"), torch.full((1,), T, device="cuda")
    t = torch.arange(T, device="cuda")
    of = torch.searchsorted(s["seq"].long(), t, right=True) - 1
    return torch.where(t < s["seq"][-1], of, torch.full_like(of, B)), (s["seq"][1:] - s["seq"][:-1]).long()


def _counts(s):
    B, E = s["c"]["B"], s["c"]["E"]
    of, _ = _seq_of(s)
    flat = (of[:, None] * E + s["idx"].long()).reshape(-1)
    return torch.bincount(flat, minlength=(B + 1) * E)[: B * E].reshape(B, E).to(torch.int32)


def _shares(s):
    """Each token's scores as shares of their sum, and d log(score) / d logit."""
    l = s["logits"]
    if s["c"]["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True), torch.ones_like(l)
    a = torch.exp(-l.abs())
    sg = torch.where(l >= 0, torch.ones_like(a), a) / (1.0 + a)
    return sg / sg.sum(1, keepdim=True), torch.where(l >= 0, a, torch.ones_like(a)) / (1.0 + a)


def _balance(s):
    c = s["c"]
    B, E, K = c["B"], c["E"], c["K"]
    of, n = _seq_of(s)
    share, slope = _shares(s)
    counts = _counts(s) if not c["grad"] else s["counts"]
    nf = n.float().clamp(min=1.0)[:, None]
    f = counts.float() * (E / K) / nf
    if not c["grad"]:
        sums = torch.zeros((B + 1, E), dtype=torch.float64, device="cuda").index_add_(0, of, share.double())[:B]
        prob = (sums / nf.double()).float()
        return {"counts": counts, "prob": prob, "loss": COEF * (f * prob).sum(1)}
    z = torch.zeros((1, E), device="cuda")
    f, w = torch.cat([f, z]), torch.cat([s["dloss"] * COEF / nf[:, 0], z[0, :1]])
    ft = f[of]
    d = w[of][:, None] * (ft - (ft * share).sum(1, keepdim=True)) * share * slope
    if s["add"] is not None:
        d = torch.where(of[:, None] < B, d + s["add"], torch.zeros_like(d))
    return {"dlogits": d}


def _encode(v, scale):
    """v / scale as E4M3 values, saturating."""
    return (v / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scale_of(amax):
    return (amax / E4M3_MAX).clamp(min=LEAST_SCALE)


def _quantize_rows(v):
    """v [rows, C] fp32 -> codes and one scale per 128 values of a row."""
    C = v.shape[1]
    b = torch.nn.functional.pad(v, (0, _blocks(C) * BLOCK - C)).reshape(v.shape[0], -1, BLOCK)
    scale = _scale_of(b.abs().amax(2))
    return _encode(b, scale[:, :, None]).reshape(v.shape[0], -1)[:, :C].contiguous(), scale


def _quantize(s):
    c, x = s["c"], s["x"].float()
    if c["form"] == "rows":
        q, scale = _quantize_rows(x)
    elif c["form"] == "squares":
        R, C = x.shape
        b = torch.nn.functional.pad(x, (0, _blocks(C) * BLOCK - C, 0, _blocks(R) * BLOCK - R))
        b = b.reshape(_blocks(R), BLOCK, _blocks(C), BLOCK)
        scale = _scale_of(b.abs().amax((1, 3)))
        q = _encode(b, scale[:, None, :, None]).reshape(_blocks(R) * BLOCK, -1)[:R, :C].contiguous()
    else:
        P, C = s["o_q"].shape
        group, at = _padded_rows(s, P)
        live = at < (s["offsets"][1:] - s["offsets"][:-1]).long()[group]
        src = (s["offsets"].long()[group] + at).clamp(max=x.shape[0] - 1)
        b = torch.where(live[:, None], x[src], torch.zeros((), device="cuda")).reshape(-1, BLOCK, C)
        scale = _scale_of(b.abs().amax(1))
        q = _encode(b, scale[:, None, :]).reshape(P, C)
        scale = scale * (torch.arange(P // BLOCK, device="cuda") * BLOCK < s["starts"][-1])[:, None]
    return {"q": q, "scale": scale}


def _f32(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _spread(scale, n, axis):
    """A scale per block of 128 along `axis` as one per element of n."""
    return scale.repeat_interleave(BLOCK, axis).narrow(axis, 0, n)


def _weights(q, scale):
    v = _f32(q)
    return v.mul_(_spread(_spread(scale, q.shape[1], 1), q.shape[2], 2))


def _pad_groups(s, v):
    """v [rows, C] -> [E, cap, C], zeros past a group's end, and the places of the live rows."""
    off, cap = s["offsets"].long(), s["cap"]
    j = torch.arange(cap, device="cuda")
    live = j[None, :] < (off[1:] - off[:-1])[:, None]
    rows = (off[:-1, None] + j[None, :]).clamp(max=v.shape[0] - 1)
    return v[rows] * live[:, :, None], rows[live], live


def _activations(s):
    return _pad_groups(s, _f32(s["a"]) * _spread(s["as"], s["a"].shape[1], 1))


def _product(s):
    a, rows, live = _activations(s)
    w = _weights(s["w"], s["ws"])
    y = a @ (w if s["c"]["transposed"] else w.transpose(1, 2))
    out = torch.empty_like(s["o"])
    out[rows] = y[live].to(out.dtype)
    return {"out": out}


def _gate_up(s):
    a, rows, live = _activations(s)
    gate = (a @ _weights(s["wg"], s["sg"]).transpose(1, 2))[live]
    up = (a @ _weights(s["wu"], s["su"]).transpose(1, 2))[live]
    q, scale = _quantize_rows(gate / (1.0 + torch.exp(-gate)) * up)
    oq, os = torch.empty_like(s["o_q"]), torch.empty_like(s["o_s"])
    oq[rows], os[rows] = q.view(torch.uint8), scale
    return {"q": oq.view(torch.float8_e4m3fn), "scale": os}


def _weight_grad(s):
    E, N, K = s["o"].shape
    cap = _blocks(s["cap"]) * BLOCK
    j = torch.arange(cap, device="cuda")
    at = s["starts"][:-1, None] + j[None, :]
    live = at < s["starts"][1:, None]
    at = at.clamp(max=s["dy"].shape[0] - 1)
    dy = (_f32(s["dy"]) * _spread(s["dys"], s["dy"].shape[0], 0))[at] * live[:, :, None]
    a = (_f32(s["a"]) * _spread(s["as"], s["a"].shape[0], 0))[at] * live[:, :, None]
    return {"dw": (dy.transpose(1, 2) @ a).to(torch.bfloat16)}


_PLAIN = {"balance": _balance, "quantize": _quantize, "product": _product, "gate_up": _gate_up,
          "weight_grad": _weight_grad}

_kept = {}


def _lib():
    """The package and the handle that a program keeps."""
    if not _kept:
        import routed_expert_ffn_04_gb300 as moe

        _kept["moe"], _kept["handle"] = moe, moe.Handle()
    return _kept["moe"], _kept["handle"]


def _own_balance(s):
    moe, h = _lib()
    c = s["c"]
    if "cfg" not in s:
        s["cfg"] = moe.make_config(c["T"], 64, c["E"], c["K"], 64, 0, 1.0)
        s["score"] = moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
        if not c["grad"]:
            size = moe.balance_loss_workspace_size(s["cfg"], num_seqs=c["B"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if c["grad"]:
        moe.balance_loss_backward(h, s["cfg"], s["logits"], s["counts"], s["dloss"], s["o_dl"], coef=COEF,
                                  score=s["score"], seq_offsets=s["seq"], dlogits_add=s["add"])
        return {"dlogits": s["o_dl"]}
    moe.balance_loss(h, s["cfg"], s["logits"], s["idx"], s["o_counts"], s["o_prob"], s["o_loss"], s["ws"], coef=COEF,
                     score=s["score"], seq_offsets=s["seq"])
    return {"counts": s["o_counts"], "prob": s["o_prob"], "loss": s["o_loss"]}


def _own_quantize(s):
    moe, h = _lib()
    if s["c"]["form"] == "columns":
        moe.quantize_fp8_columns(h, s["x"], s["offsets"], s["o_q"], s["o_s"], num_groups=s["c"]["E"])
    else:
        moe.quantize_fp8(h, s["x"], s["o_q"], s["o_s"], squares=s["c"]["form"] == "squares")
    return {"q": s["o_q"].view(torch.float8_e4m3fn), "scale": s["o_s"]}


def _own_product(s):
    moe, h = _lib()
    c = s["c"]
    moe.grouped_gemm_fp8(h, s["a"], s["as"], s["offsets"], s["w"], s["ws"], s["o"], num_groups=c["E"], N=c["N"],
                         K=c["K"], transposed=c["transposed"])
    return {"out": s["o"]}


def _own_gate_up(s):
    moe, h = _lib()
    c = s["c"]
    moe.grouped_gate_up_fp8(h, s["a"], s["as"], s["offsets"], s["wg"], s["sg"], s["wu"], s["su"], s["o_q"], s["o_s"],
                            num_groups=c["E"], H=c["H"], I=c["I"])
    return {"q": s["o_q"].view(torch.float8_e4m3fn), "scale": s["o_s"]}


def _own_weight_grad(s):
    moe, h = _lib()
    c = s["c"]
    moe.grouped_weight_grad_fp8(h, s["dy"], s["dys"], s["a"], s["as"], s["offsets"], s["o"], rows=c["T"] * c["top"],
                                num_groups=c["E"], N=c["N"], K=c["K"])
    return {"dw": s["o"]}


_OWN = {"balance": _own_balance, "quantize": _own_quantize, "product": _own_product, "gate_up": _own_gate_up,
        "weight_grad": _own_weight_grad}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "balance":
        n, BE = c["T"] * c["E"], c["B"] * c["E"]
        if c["grad"]:
            return {"bytes": 4 * n * (3 if c["add"] else 2) + 4 * BE + 4 * c["B"], "flops": 8 * n}
        return {"bytes": 4 * n + 4 * c["T"] * c["K"] + 8 * BE + 4 * c["B"], "flops": 6 * n}
    if c["op"] == "quantize":
        b = 2 if c["x"] == "bf16" else 4
        if c["form"] == "columns":
            n = c["T"] * c["K"] * c["C"]
            return {"bytes": n * (b + 1) + 4 * (n // BLOCK) + 4 * (c["E"] + 1), "flops": 3 * n}
        n = c["rows"] * c["C"]
        blocks = (c["rows"] if c["form"] == "rows" else _blocks(c["rows"])) * _blocks(c["C"])
        return {"bytes": n * (b + 1) + 4 * blocks, "flops": 3 * n}
    R = c["T"] * c["top"]
    G = min(c["E"], R)  # groups that can have rows
    if c["op"] == "gate_up":
        H, I = c["H"], c["I"]
        return {"bytes": 2 * G * H * I + R * (H + 4 * _blocks(H)) + R * (I + 4 * _blocks(I)) + 4 * (c["E"] + 1),
                "flops": 4 * R * H * I}
    N, K = c["N"], c["K"]
    if c["op"] == "product":
        return {"bytes": G * N * K + R * (K + 4 * _blocks(K)) + R * N * (2 if c["out"] == "bf16" else 4)
                + 4 * (c["E"] + 1), "flops": 2 * R * N * K}
    return {"bytes": R * (N + K) + 4 * (R // BLOCK) * (N + K) + 2 * c["E"] * N * K + 4 * (c["E"] + 1),
            "flops": 2 * R * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: t.to(torch.float64)  # noqa: E731
    c, op = case, case["op"]
    if op == "balance":
        T, E, B, K = c["T"], c["E"], c["B"], c["K"]
        ends = s["seq"].tolist() if s["seq"] is not None else [0, T]
        x = d(s["logits"])
        logs = x if c["score"] == "softmax" else torch.nn.functional.logsigmoid(x)
        share = torch.exp(logs - torch.logsumexp(logs, 1, keepdim=True))
        slope = torch.ones_like(x) if c["score"] == "softmax" else torch.special.expit(-x)
        counts = torch.zeros((B, E), dtype=torch.int32, device="cuda")
        prob = torch.zeros((B, E), dtype=torch.float64, device="cuda")
        loss = torch.zeros((B,), dtype=torch.float64, device="cuda")
        dl = torch.zeros_like(x)
        for b in range(B):
            lo, hi = ends[b], ends[b + 1]
            if lo == hi:
                continue
            n = hi - lo
            counts[b] = torch.histc(s["idx"][lo:hi].double(), bins=E, min=-0.5, max=E - 0.5).int()
            load = d(counts[b]) * E / (K * n)
            prob[b] = share[lo:hi].sum(0) / n
            loss[b] = COEF * torch.dot(load, prob[b])
            if c["grad"]:
                mean = torch.mv(share[lo:hi], load)
                dl[lo:hi] = share[lo:hi] * slope[lo:hi] * (load - mean[:, None]) * (d(s["dloss"][b]) * COEF / n)
                if s["add"] is not None:
                    dl[lo:hi] += d(s["add"][lo:hi])
        return {"dlogits": dl} if c["grad"] else {"counts": counts, "prob": prob, "loss": loss}
    if op == "quantize":
        x = d(s["x"])
        if c["form"] != "columns":
            h = 1 if c["form"] == "rows" else BLOCK
            q, scale = _quantize64(x, h, BLOCK)
            return {"q": q, "scale": scale}
        q = torch.zeros(s["o_q"].shape, dtype=torch.float64, device="cuda")
        scale = torch.zeros(s["o_s"].shape, dtype=torch.float64, device="cuda")
        off, at = s["offsets"].tolist(), s["starts"].tolist()
        for e in range(c["E"]):
            n = off[e + 1] - off[e]
            if n:
                qe, se = _quantize64(x[off[e]:off[e + 1]], BLOCK, 1)
                q[at[e]:at[e] + n] = qe
                scale[at[e] // BLOCK:at[e + 1] // BLOCK] = se
        return {"q": q, "scale": scale}
    f8 = lambda t: t.view(torch.float8_e4m3fn).to(torch.float64)  # noqa: E731
    up = lambda t, n, axis: torch.repeat_interleave(d(t), BLOCK, dim=axis).narrow(axis, 0, n)  # noqa: E731
    off, at = s["offsets"].tolist(), s["starts"].tolist()
    square = lambda q, sc: f8(q) * up(up(sc, q.shape[0], 0), q.shape[1], 1)  # noqa: E731
    if op == "weight_grad":
        dw = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            lo, hi = at[e], at[e + 1]
            if lo < hi:
                l, r = (f8(s[n][lo:hi]) * up(s[n + "s"][lo // BLOCK:hi // BLOCK], hi - lo, 0) for n in ("dy", "a"))
                dw[e] = torch.mm(l.t(), r)
        return {"dw": dw}
    rows = s["a"].shape[0]
    if op == "product":
        out = torch.zeros((rows, c["N"]), dtype=torch.float64, device="cuda")
    else:
        q = torch.zeros((rows, c["I"]), dtype=torch.float64, device="cuda")
        scale = torch.zeros((rows, _blocks(c["I"])), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        x = f8(s["a"][lo:hi]) * up(s["as"][lo:hi], s["a"].shape[1], 1)
        if op == "product":
            w = square(s["w"][e], s["ws"][e])
            out[lo:hi] = torch.mm(x, w if c["transposed"] else w.t())
        else:
            gate, u = (torch.mm(x, square(s["w" + n][e], s["s" + n][e]).t()) for n in ("g", "u"))
            q[lo:hi], scale[lo:hi] = _quantize64(gate * torch.special.expit(gate) * u, 1, BLOCK)
    return {"out": out} if op == "product" else {"q": q, "scale": scale}


def _quantize64(x, height, width):
    """Codes as values and scales of blocks of height x width."""
    R, C = x.shape
    nr, nc = -(-R // height), -(-C // width)
    full = torch.zeros((nr * height, nc * width), dtype=torch.float64, device=x.device)
    full[:R, :C] = x
    tiles = full.unflatten(1, (nc, width)).unflatten(0, (nr, height))
    scale = torch.clamp(torch.linalg.vector_norm(tiles, ord=math.inf, dim=(1, 3)) / E4M3_MAX, min=LEAST_SCALE)
    q = _e4m3(tiles / scale[:, None, :, None]).reshape(nr * height, nc * width)
    return q[:R, :C].contiguous(), scale


def _e4m3(v):
    """Nearest E4M3 number (ties to even), saturating at 448."""
    a = v.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)
