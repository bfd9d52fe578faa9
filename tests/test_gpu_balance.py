"""Balance loss of the router and its gradient against the definition in 64 bits.

Tolerances. exp, the quotient and the sum of E scores in fp32: a share is off by at most (E / 32 + 16) 2^-23 of itself
(five levels of a shuffle sum, E / 32 additions per lane, exp.approx with an argument rounded at |x| <= 16: |x| 2^-24 +
2^-22, the quotient 2^-22). Sums over tokens add at most their number of additions in a row times 2^-24."""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe

pytestmark = pytest.mark.gpu

F32, F64, I32 = torch.float32, torch.float64, torch.int32
SCORES = {"sigmoid": moe.MOE_SCORE_SIGMOID, "softmax": moe.MOE_SCORE_SOFTMAX}


@pytest.fixture(scope="module")
def handle():
    h = moe.Handle(0)
    yield h
    h.close()


def cfg_of(T, E, K):
    return moe.make_config(T, 64, E, K, 64, 0, 1.0)


def shares64(x, score):
    logs = x if score == "softmax" else torch.nn.functional.logsigmoid(x)
    p = torch.softmax(logs, 1)
    return torch.where(torch.isneginf(x).all(1, keepdim=True), torch.zeros_like(p), p)


def reference(logits, idx, ends, score, coef, E, K):
    x, B = logits.to(F64), len(ends) - 1
    p = shares64(x, score)
    counts = torch.zeros((B, E), dtype=I32, device="cuda")
    prob, loss = torch.zeros((B, E), dtype=F64, device="cuda"), torch.zeros(B, dtype=F64, device="cuda")
    for b in range(B):
        lo, hi = ends[b], ends[b + 1]
        if hi > lo:
            flat = idx[lo:hi].reshape(-1).long()
            counts[b] = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
            prob[b] = p[lo:hi].mean(0)
            loss[b] = coef * (counts[b].to(F64) * E / (K * (hi - lo)) * prob[b]).sum()
    return counts, prob, loss


def run(handle, logits, idx, ends, score, coef, E, K):
    T, B = logits.shape[0], len(ends) - 1
    cfg = cfg_of(T, E, K)
    seq = None if ends == [0, T] else torch.tensor(ends, dtype=I32, device="cuda")
    counts, prob = torch.full((B, E), -7, dtype=I32, device="cuda"), torch.full((B, E), -7.0, device="cuda")
    loss = torch.full((B,), -7.0, device="cuda")
    ws = torch.full((moe.balance_loss_workspace_size(cfg, B),), 0xA5, dtype=torch.uint8, device="cuda")
    moe.balance_loss(handle, cfg, logits, idx, counts, prob, loss, ws, coef=coef, score=SCORES[score], seq_offsets=seq)
    return cfg, seq, counts, prob, loss


def problem(T, E, K, seed=0, bias=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((T, E), device="cuda", generator=g) + bias * torch.randn((1, E), device="cuda", generator=g)
    return logits, torch.topk(logits, K, dim=1).indices.to(I32), g


def share_tol(E):
    return (E / 32 + 16) * 2.0 ** -23


def grad64(logits, counts, ends, dloss, score, coef, E, K):
    x, p = logits.to(F64), shares64(logits.to(F64), score)
    d = torch.zeros_like(x)
    for b in range(len(ends) - 1):
        lo, hi = ends[b], ends[b + 1]
        if hi > lo:
            f = counts[b].to(F64) * E / (K * (hi - lo))
            q = p[lo:hi]
            d[lo:hi] = float(dloss[b]) * coef / (hi - lo) * (f - (q * f).sum(1, keepdim=True)) * q
            if score == "sigmoid":
                d[lo:hi] *= torch.sigmoid(-x[lo:hi])
    return d


CASES = [(1, 8, 2, [0, 1]), (1, 1, 1, [0, 1]), (17, 64, 6, [0, 17]), (61, 192, 8, [0, 61]), (1000, 192, 8, [0, 1000]), (333, 33, 5, [0, 333]),
         (700, 256, 8, [0, 0, 1, 33, 33, 64, 640, 690]), (96, 1024, 32, [5, 40, 96]), (40, 512, 3, [0, 13, 40]), (3000, 100, 4, [0, 3000]),
         (20000, 65, 1, [0, 9999, 20000]), (300, 16, 2, list(range(0, 301, 3))),
         (6, 24, 1, [0, 0, 0, 2] + [3] * 40 + [6] * 40), (84, 56, 3, sorted((i * 37) % 80 for i in range(64))),
         (9001, 4, 2, [i * i * 2 for i in range(65)] + [9001]), (5000, 128, 8, [0, 0, 1, 2, 40, 41, 3000, 3000, 3001, 4990])]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T, E, K, ends", CASES)
def test_loss(handle, T, E, K, ends, score):
    logits, idx, _ = problem(T, E, K)
    _, _, counts, prob, loss = run(handle, logits, idx, ends, score, 0.25, E, K)
    rc, rp, rl = reference(logits, idx, ends, score, 0.25, E, K)
    assert torch.equal(counts, rc)
    tol = share_tol(E) + (T / 512 + 64) * 2.0 ** -24  # a warp's tokens in a row, then warps, strips
    assert ((prob.to(F64) - rp).abs() <= tol * rp).all()
    assert ((loss.to(F64) - rl).abs() <= (tol + (E / 32 + 16) * 2.0 ** -24) * rl).all()
    assert handle.device_status() == 0


@pytest.mark.parametrize("add", [None, "new", "same"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T, E, K, ends", CASES)
def test_gradient(handle, T, E, K, ends, score, add):
    logits, idx, g = problem(T, E, K, seed=1)
    B = len(ends) - 1
    cfg, seq, counts, _, _ = run(handle, logits, idx, ends, score, 0.25, E, K)
    dloss = torch.rand(B, device="cuda", generator=g) + 0.5
    want = grad64(logits, counts, ends, dloss, score, 0.25, E, K)
    dl = torch.full((T, E), 7.0, device="cuda")
    extra = None
    if add:
        extra = 1e-3 * torch.randn((T, E), device="cuda", generator=g)
        if add == "same":
            dl = extra.clone()
    before = dl.clone()
    moe.balance_loss_backward(handle, cfg, logits, counts, dloss, dl, coef=0.25, score=SCORES[score], seq_offsets=seq,
                              dlogits_add=None if add is None else dl if add == "same" else extra)
    f = torch.zeros((T, 1), dtype=F64, device="cuda")  # the largest of |f| and its mean: what the difference is taken of
    scale = torch.zeros((T, 1), dtype=F64, device="cuda")
    for b in range(B):
        lo, hi = ends[b], ends[b + 1]
        if hi > lo:
            f[lo:hi] = counts[b].max().double() * E / (K * (hi - lo))
            scale[lo:hi] = float(dloss[b]) * 0.25 / (hi - lo)
    p = shares64(logits.to(F64), score)
    tol = scale * f * p * (2 * share_tol(E) + 2.0 ** -20)
    if extra is not None:
        want = want + extra.to(F64)
        tol = tol + 2.0 ** -24 * want.abs()
    err = (dl.to(F64) - want).abs()[ends[0]:ends[-1]]
    assert (err <= tol[ends[0]:ends[-1]] + 1e-30).all()
    assert torch.equal(dl[:ends[0]], before[:ends[0]]) and torch.equal(dl[ends[-1]:], before[ends[-1]:])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_against_differences(handle, score):
    T, E, K = 24, 16, 3
    logits, idx, _ = problem(T, E, K, seed=2)
    cfg, _, counts, _, _ = run(handle, logits, idx, [0, T], score, 1.0, E, K)
    dl = torch.empty((T, E), device="cuda")
    moe.balance_loss_backward(handle, cfg, logits, counts, torch.ones(1, device="cuda"), dl, score=SCORES[score])
    f = counts[0].to(F64) * E / (K * T)
    loss = lambda x: (shares64(x, score).mean(0) * f).sum()  # noqa: E731
    for t, e in ((0, 0), (5, 7), (23, 15)):
        d = torch.zeros((T, E), dtype=F64, device="cuda")
        d[t, e] = 1e-4
        x = logits.to(F64)
        assert abs(float(loss(x + d) - loss(x - d)) / 2e-4 - float(dl[t, e])) <= 1e-6 * float(f.max()) / T * 10


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_experts(handle, score):
    """Experts masked by -infinity or the lowest value, rows that leave nothing, scores that all underflow."""
    T, E, K = 50, 48, 4
    logits, idx, _ = problem(T, E, K, seed=3)
    logits[:, 5] = float("-inf")
    logits[:, 6] = torch.finfo(F32).min
    logits[3] = float("-inf")
    logits[4] = torch.finfo(F32).min
    logits[5] -= 200.0
    logits[6, 1:] = float("-inf")
    if score == "sigmoid":
        logits[7, 2] = float("inf")
    cfg, _, counts, prob, loss = run(handle, logits, idx, [0, T], score, 1.0, E, K)
    rc, rp, rl = reference(logits, idx, [0, T], score, 1.0, E, K)
    assert torch.equal(counts, rc)
    # row 5: exp of logits near -200, rounded there to 2^-17 of themselves
    assert ((prob.to(F64) - rp).abs() <= 1e-6 * rp + 2.0 ** -16 / T).all() and abs(float(loss[0]) - float(rl[0])) <= 1e-5 * float(rl[0])
    dl = torch.full((T, E), 7.0, device="cuda")
    moe.balance_loss_backward(handle, cfg, logits, counts, torch.ones(1, device="cuda"), dl, score=SCORES[score])
    want = grad64(logits, counts, [0, T], [1.0], score, 1.0, E, K).nan_to_num(0.0)  # 64 bits: inf * 0 of masked logits
    assert dl.isfinite().all() and (dl[torch.isneginf(logits)] == 0).all()
    fmax = float(counts.max()) * E / (K * T)
    assert ((dl.to(F64) - want).abs() <= fmax / T * 2.0 ** -15).all()


def test_nan_logit_stays_in_its_sequence(handle):
    T, E, K, ends = 64, 32, 2, [0, 20, 64]
    logits, idx, _ = problem(T, E, K, seed=4)
    logits[30, 3] = float("nan")
    cfg, seq, counts, prob, loss = run(handle, logits, idx, ends, "sigmoid", 1.0, E, K)
    assert prob[0].isfinite().all() and prob[1].isnan().all() and loss.isnan().tolist() == [False, True]
    dl = torch.empty((T, E), device="cuda")
    moe.balance_loss_backward(handle, cfg, logits, counts, torch.ones(2, device="cuda"), dl, seq_offsets=seq)
    assert dl.isnan().any(1).nonzero().flatten().tolist() == [30]


def test_ids_out_of_range_and_twice(handle):
    T, E, K = 10, 8, 3
    logits, idx, _ = problem(T, E, K, seed=5)
    idx[2, 1], idx[3, 0], idx[4] = -1, E, 2
    _, _, counts, _, _ = run(handle, logits, idx, [0, T], "sigmoid", 1.0, E, K)
    assert torch.equal(counts, reference(logits, idx, [0, T], "sigmoid", 1.0, E, K)[0])
    assert handle.device_status() == 16 and handle.device_status() == 0  # MOE_DEV_BAD_EXPERT_ID, then cleared


def test_no_tokens(handle):
    logits, idx = torch.empty((0, 8), device="cuda"), torch.empty((0, 2), dtype=I32, device="cuda")
    cfg, _, counts, prob, loss = run(handle, logits, idx, [0, 0], "sigmoid", 1.0, 8, 2)
    assert (counts == 0).all() and (prob == 0).all() and (loss == 0).all()
    moe.balance_loss_backward(handle, cfg, logits, counts, torch.ones(1, device="cuda"), torch.empty_like(logits))


def test_same_bits_streams_graph(handle):
    T, E, K, ends = 5000, 192, 8, [0, 1234, 1234, 4999]
    logits, idx, _ = problem(T, E, K, seed=6)
    first = run(handle, logits, idx, ends, "sigmoid", 1.0, E, K)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        other = run(handle, logits, idx, ends, "sigmoid", 1.0, E, K)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[2:], other[2:]))
    cfg, seq, counts, prob, loss = first
    ws = torch.empty(moe.balance_loss_workspace_size(cfg, 3), dtype=torch.uint8, device="cuda")
    out = [torch.zeros_like(t) for t in (counts, prob, loss)]
    dl, dloss = torch.zeros((T, E), device="cuda"), torch.ones(3, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.balance_loss(handle, cfg, logits, idx, *out, ws, seq_offsets=seq)
        moe.balance_loss_backward(handle, cfg, logits, out[0], dloss, dl, seq_offsets=seq)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[2:], out))
    want = torch.zeros_like(dl)
    moe.balance_loss_backward(handle, cfg, logits, counts, dloss, want, seq_offsets=seq)
    assert torch.equal(dl, want)
