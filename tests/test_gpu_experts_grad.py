"""moe_grouped_swiglu_backward against the formulas in 64 bits.

Tolerances: h, dgate and dup are rounded to bf16 (2^-8) before the products that read them, and each output once more.
So every element may be off by 2^-8 of its own size plus 2^-8 of the product of the absolute values (fp32 accumulation
adds K * 2^-24 of that: inside the 1.1 below for K <= 3000), and the 2-norm of an output, over which independent
roundings (rms 2^-8 / sqrt(3) = 2.3e-3 at most, two of them) average, by at most 5e-3 of its norm.
"""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe

pytestmark = pytest.mark.gpu
B = 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load(build_if_missing=True)
    return moe.Handle(0)


def _randn(g, shape, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(BF)


def _problem(counts, H, I, lead=0, trail=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = [lead]
    for c in counts:
        off.append(off[-1] + c)
    rows, G = off[-1] + trail, len(counts)
    return dict(off=off, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), a=_randn(g, (rows, H)),
                dy=_randn(g, (rows, H), 0.05), wg=_randn(g, (G, I, H), 1.5 * H ** -0.5),
                wu=_randn(g, (G, I, H), 1.5 * H ** -0.5), wd=_randn(g, (G, H, I), I ** -0.5), H=H, I=I, G=G, rows=rows)


def _run(handle, p, want=("da", "dw"), offsets=True, ws_fill=0xFF):
    shape = lambda k: torch.full_like(p[k], 7.0)  # noqa: E731
    o = dict(da=shape("a"), dg=shape("wg"), du=shape("wu"), dd=shape("wd"))
    ws = torch.full((moe.grouped_gemm_backward_workspace_size(p["rows"], p["H"], p["I"], num_groups=p["G"]),), ws_fill,
                    dtype=torch.uint8, device="cuda")
    dws = [o["dg"], o["du"], o["dd"]] if "dw" in want else [None] * 3
    moe.grouped_swiglu_backward(handle, p["a"], p["dy"], p["offsets"] if offsets else None, p["wg"], p["wu"], p["wd"],
                                o["da"] if "da" in want else None, *dws, ws, num_groups=p["G"], H=p["H"], I=p["I"])
    assert handle.device_status() == 0
    return o


def _check(got, ref, size, what):
    err = (got.double() - ref).abs()
    assert (err <= 1.02 * B * ref.abs() + 1.1 * B * size).all(), (what, err.max().item())
    n = ref.norm()
    assert n == 0 or (got.double() - ref).norm() <= 5e-3 * n, (what, ((got.double() - ref).norm() / n).item())


def _against_formulas(p, o):
    for e in range(p["G"]):
        b, n = p["off"][e], p["off"][e + 1]
        if b == n:
            assert (o["dg"][e] == 0).all() and (o["du"][e] == 0).all() and (o["dd"][e] == 0).all()
            continue
        x, dy, wg, wu, wd = (t.double() for t in (p["a"][b:n], p["dy"][b:n], p["wg"][e], p["wu"][e], p["wd"][e]))
        gate, up, q = x @ wg.T, x @ wu.T, dy @ wd
        sg = torch.sigmoid(gate)
        h, dg, du = gate * sg * up, q * up * sg * (1 + gate * (1 - sg)), q * gate * sg
        _check(o["dd"][e], dy.T @ h, dy.abs().T @ h.abs(), f"dw_down {e}")
        _check(o["dg"][e], dg.T @ x, dg.abs().T @ x.abs(), f"dw_gate {e}")
        _check(o["du"][e], du.T @ x, du.abs().T @ x.abs(), f"dw_up {e}")
        _check(o["da"][b:n], dg @ wg + du @ wu, dg.abs() @ wg.abs() + du.abs() @ wu.abs(), f"da {e}")
    assert (o["da"][:p["off"][0]] == 7.0).all() and (o["da"][p["off"][-1]:] == 7.0).all()  # rows of no group


RAGGED = [0, 1, 15, 16, 17, 31, 33, 0, 0, 63, 64, 65, 127, 128, 129, 300, 0]


@pytest.mark.parametrize("counts,H,I,lead,trail", [
    ([1], 64, 64, 0, 0), ([5], 128, 64, 0, 0), ([130], 64, 192, 0, 0), ([16, 16], 320, 128, 0, 0),
    (RAGGED, 128, 192, 0, 0), (RAGGED, 192, 320, 3, 40), (RAGGED[::-1], 512, 256, 0, 7), ([0, 0, 0], 64, 64, 0, 9),
    ([700, 3, 0, 257], 1024, 576, 1, 0), ([2] * 200, 256, 128, 0, 0), ([0] * 300 + [40] + [0] * 700, 64, 128, 0, 0),
    ([341, 320], 4096, 1536, 0, 0),
])
def test_against_formulas(handle, counts, H, I, lead, trail):
    p = _problem(counts, H, I, lead, trail)
    o = _run(handle, p)
    _against_formulas(p, o)
    again = _run(handle, p, ws_fill=0)
    for k in o:
        assert torch.equal(o[k], again[k]), k
    only = _run(handle, p, want=("da",))
    assert torch.equal(only["da"], o["da"]) and (only["dg"] == 7.0).all()
    only = _run(handle, p, want=("dw",))
    assert all(torch.equal(only[k], o[k]) for k in ("dg", "du", "dd")) and (only["da"] == 7.0).all()


@pytest.mark.parametrize("rows", [1, 63, 64, 200, 1030])
def test_one_group_without_offsets(handle, rows):
    p = _problem([rows], 256, 320)
    o, d = _run(handle, p), _run(handle, p, offsets=False)
    _against_formulas(p, o)
    for k in o:
        assert torch.equal(o[k], d[k]), k


def test_a_groups_infinities_and_nans_stay_in_it(handle):
    """The stages that hold a group's last rows also load the next group's: nothing of them may get in."""
    p = _problem([37, 90, 5, 64, 3], 192, 128, lead=2, trail=5)
    clean = _run(handle, p)
    bad = dict(p, a=p["a"].clone(), dy=p["dy"].clone())
    for b, n in ((0, 2), (39, 129), (198, 201), (201, 206)):  # before, group 1, group 4, after
        bad["a"][b:n] = float("inf")
        bad["dy"][b:n] = float("nan")
    o = _run(handle, bad)
    for e, (b, n) in ((0, (2, 39)), (2, (129, 134)), (3, (134, 198))):
        assert torch.equal(o["da"][b:n], clean["da"][b:n])
        for k in ("dg", "du", "dd"):
            assert torch.equal(o[k][e], clean[k][e]), (k, e)
    assert o["dg"][1].isnan().any()


def test_no_rows(handle):
    p = _problem([0, 0], 64, 64)
    p["a"] = p["dy"] = torch.empty((0, 64), dtype=BF, device="cuda")
    o = _run(handle, p)
    assert all((o[k] == 0).all() for k in ("dg", "du", "dd"))


def test_against_differences(handle):
    """Directional derivatives of sum(dy * y) in 64 bits. The gradient's own roundings (about 2^-8 an element, of
    random sign) add up like a random walk: 4 standard deviations of rms 3.2e-3 a term."""
    counts, H, I = [40, 0, 25], 128, 192
    p = _problem(counts, H, I)
    o = _run(handle, p)

    def loss(a, wg, wu, wd):
        t = 0
        for e in range(3):
            b, n = p["off"][e], p["off"][e + 1]
            g, u = a[b:n] @ wg[e].T, a[b:n] @ wu[e].T
            t = t + (p["dy"][b:n].double() * ((g * torch.sigmoid(g) * u) @ wd[e].T)).sum()
        return t

    base = [p[k].double() for k in ("a", "wg", "wu", "wd")]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for i, k in enumerate(("da", "dg", "du", "dd")):
        v = torch.randn(base[i].shape, device="cuda", generator=gen, dtype=torch.float64) * base[i].std()
        t = 1e-4
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + t * v, base[i] - t * v
        dif = (loss(*up) - loss(*dn)) / (2 * t)
        terms = o[k].double() * v
        assert (terms.sum() - dif).abs() <= 4 * 3.2e-3 * terms.norm() + 1e-6 * terms.abs().sum(), k


def test_the_forwards_own_result(handle):
    """The recomputed h is the forward's: y from moe_grouped_swiglu_gemm, and dw_down = dy^T h, agree with one h."""
    p = _problem([70, 33], 256, 128)
    y = torch.empty((p["rows"], 256), device="cuda")
    ws = torch.empty(moe.grouped_gemm_workspace_size(p["rows"], 256, 128, num_groups=2), dtype=torch.uint8, device="cuda")
    moe.grouped_swiglu_gemm(handle, p["a"], p["offsets"], p["wg"], p["wu"], p["wd"], y, ws, num_groups=2, H=256, I=128)
    o = _run(handle, p)
    for e in range(2):  # <y, dy> = <dw_down, w_down>: both are sum_r dy_r W_d h_r
        b, n = p["off"][e], p["off"][e + 1]
        lhs = (y[b:n].double() * p["dy"][b:n].double()).sum()
        terms = o["dd"][e].double() * p["wd"][e].double()
        assert (lhs - terms.sum()).abs() <= 4 * 3.2e-3 * terms.norm() + 4 * 3.2e-3 * (y[b:n] * p["dy"][b:n].float()).double().norm()


def test_refusals(handle):
    p = _problem([20, 12], 128, 64)
    ws = torch.empty(moe.grouped_gemm_backward_workspace_size(32, 128, 64, num_groups=2), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(p[k]) for k in ("a", "wg", "wu", "wd")]

    def call(**kw):
        d = dict(a=p["a"], dy=p["dy"], offsets=p["offsets"], wg=p["wg"], wu=p["wu"], wd=p["wd"], da=out[0], dg=out[1],
                 du=out[2], dd=out[3], ws=ws, num_groups=2, H=128, I=64, dtype=moe.MOE_BF16)
        d.update(kw)
        moe.grouped_swiglu_backward(handle, d["a"], d["dy"], d["offsets"], d["wg"], d["wu"], d["wd"], d["da"], d["dg"],
                                    d["du"], d["dd"], d["ws"], num_groups=d["num_groups"], H=d["H"], I=d["I"],
                                    dtype=d["dtype"])

    call()
    inv = moe.MOE_ERR_INVALID_ARG
    for kw, st in ((dict(dg=None), inv), (dict(da=None, dg=None, du=None, dd=None), inv), (dict(offsets=None), inv),
                   (dict(dy=p["dy"][:31]), inv), (dict(a=p["a"].float()), inv), (dict(wd=p["wd"].transpose(1, 2)), inv),
                   (dict(da=out[0].cpu()), inv), (dict(I=32), inv), (dict(H=64), inv),
                   (dict(dtype=moe.MOE_MXFP8_E4M3), moe.MOE_ERR_UNSUPPORTED), (dict(dtype=9), inv),
                   (dict(ws=ws[:ws.numel() - 256]), moe.MOE_ERR_WORKSPACE)):
        with pytest.raises(moe.MoEError) as e:
            call(**kw)
        assert e.value.status == st, kw
    assert handle.device_status() == 0


def test_chunks_of_every_height_over_many_launches(handle):
    """Every multiple of 32 rows as a chunk (alone and beside a larger one), long reductions, many launches: each of the
    roles that fill a stage has to have a part in it, or it may fall a ring behind."""
    p = _problem([32, 64, 96, 128, 160, 192, 224, 256, 288, 512, 545, 128, 128], 2048, 1024)
    o = _run(handle, p)
    _against_formulas(p, o)
    for _ in range(40):
        again = _run(handle, p)
        for k in o:
            assert torch.equal(o[k], again[k]), k


def test_two_streams_at_once(handle):
    """Chains of launches on two streams, with workspaces of their own, share the GPU and keep their results."""
    ps = [_problem([100, 0, 300, 41], 512, 256, seed=1), _problem([31, 64, 7], 1024, 192, seed=2)]
    want = [_run(handle, p) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    bufs = []
    for p in ps:
        size = moe.grouped_gemm_backward_workspace_size(p["rows"], p["H"], p["I"], num_groups=p["G"])
        bufs.append([torch.empty_like(p[k]) for k in ("a", "wg", "wu", "wd")] +
                    [torch.empty(size, dtype=torch.uint8, device="cuda")])
    torch.cuda.synchronize()
    for _ in range(30):
        for p, b, s in zip(ps, bufs, streams):
            moe.grouped_swiglu_backward(handle, p["a"], p["dy"], p["offsets"], p["wg"], p["wu"], p["wd"], *b,
                                        num_groups=p["G"], H=p["H"], I=p["I"], stream=s)
    torch.cuda.synchronize()
    assert handle.device_status() == 0
    for w, b in zip(want, bufs):
        for k, t in zip(("da", "dg", "du", "dd"), b):
            assert torch.equal(w[k], t), k


def test_operands_written_by_the_launch_just_before(handle):
    """The chained launches read nothing before the launch ahead of them has ended: each operand in turn is the last one
    written, `a` by one of the library's own dependent launches."""
    ps = [_problem([100, 0, 300, 41], 512, 256, seed=1), _problem([7, 250, 3, 181], 512, 256, seed=2)]
    rows, names = ps[0]["rows"], ["offsets", "a", "dy", "wg", "wu", "wd"]
    want = [_run(handle, p) for p in ps]
    b = {k: ps[0][k].clone() for k in names}
    out = [torch.empty_like(ps[0][k]) for k in ("a", "wg", "wu", "wd")]
    ws = torch.empty(moe.grouped_gemm_backward_workspace_size(rows, 512, 256, num_groups=4), dtype=torch.uint8, device="cuda")
    cfg, same = moe.make_config(rows, 512, 4, 1, 64, 0, 1.0), torch.arange(rows, dtype=torch.int32, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(48):
        p = ps[i & 1]
        at = (i >> 1) % len(names)
        for k in names[at + 1:] + names[:at + 1]:
            if k == "a":  # one row per token: a copy
                moe.permute_backward(handle, cfg, p["a"], same, b["a"])
            else:
                torch.mul(p[k], 1, out=b[k])
        moe.grouped_swiglu_backward(handle, *[b[k] for k in ("a", "dy", "offsets", "wg", "wu", "wd")], *out, ws,
                                    num_groups=4, H=512, I=256)
        for k, t in zip(("da", "dg", "du", "dd"), out):
            wrong += (t != want[i & 1][k]).sum()
    assert wrong.item() == 0 and handle.device_status() == 0


@pytest.mark.parametrize("counts,H,I,groups", [
    ([37, 3], 192, 128, (0, 1)), ([17, 3], 128, 64, (0, 1)), ([5, 90, 0, 0], 640, 320, (1,)), ([16, 32, 1, 1, 1], 64, 192, (2, 3, 4)),
    ([401], 320, 576, (0,)), ([1], 64, 64, (0,)),
])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", [("dy",), ("a",), ("a", "dy")])
def test_rows_of_no_group_stay_out(handle, counts, H, I, groups, bad, where):
    """Rows before the first group and after the last one may hold anything. `groups`: those whose last step of 16 rows
    reaches past the last group's end."""
    p = _problem(counts, H, I, lead=4, trail=20)
    assert all((p["off"][e] + (counts[e] + 15) // 16 * 16 > p["off"][-1]) == (e in groups) for e in range(len(counts)) if counts[e])
    clean = _run(handle, p)
    _against_formulas(p, clean)
    q = dict(p)
    for k in where:
        q[k] = p[k].clone()
        q[k][:4] = bad
        q[k][p["off"][-1]:] = bad
    o = _run(handle, q)
    for k in o:
        assert torch.equal(o[k], clean[k]), k


def test_dropped_pairs_leave_nothing_in_the_weights(handle):
    """The rows of dropped pairs, which the combine's gradient does not write, lie after the last group."""
    T, H, E, K, I = 50, 128, 6, 2, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    cfg = moe.make_config(T, H, E, K, I, 0, 1.5)
    logits = torch.randn((T, E), device="cuda", generator=g)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    idx, tw = i32((T, K)), torch.empty((T, K), device="cuda")
    moe.route(handle, cfg, logits, idx, tw)
    sent = idx.clone()
    sent.view(-1)[torch.randperm(T * K, device="cuda", generator=g)[:21]] = E + 5
    counts, offsets, perm, f2p = i32(E), i32(E + 1), i32(T * K), i32(T * K)
    x, xp = _randn(g, (T, H)), torch.zeros((T * K, H), dtype=BF, device="cuda")
    ws = torch.empty(moe.permute_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    moe.permute(handle, cfg, x, sent, counts, offsets, perm, f2p, xp, ws)
    assert handle.device_status() != 0  # the dropped pairs are reported
    off = offsets.tolist()
    assert off[-1] == T * K - 21
    y, dout = torch.randn((T * K, H), device="cuda", generator=g), _randn(g, (T, H))
    p = dict(off=off, offsets=offsets, a=xp, wg=_randn(g, (E, I, H), 0.1), wu=_randn(g, (E, I, H), 0.1),
             wd=_randn(g, (E, H, I), 0.1), H=H, I=I, G=E, rows=T * K)
    got = []
    for fill in (0.0, float("nan")):
        dy, dtw = torch.full((T * K, H), fill, dtype=BF, device="cuda"), torch.empty((T, K), device="cuda")
        moe.combine_backward(handle, cfg, dout, y, tw, f2p, dy, dtw)
        got.append(_run(handle, dict(p, dy=dy)))
    for k in got[0]:
        assert torch.equal(got[0][k], got[1][k]), k


@pytest.mark.parametrize("groups,offsets", [(2, True), (1, True), (1, False)])
def test_no_rows_and_no_weight_gradients(handle, groups, offsets):
    """A step without rows under frozen weights: the only output asked for has no elements."""
    p = _problem([0] * groups, 64, 128)
    o = _run(handle, p, want=("da",), offsets=offsets)
    assert o["da"].shape == (0, 64) and all((o[k] == 7.0).all() for k in ("dg", "du", "dd"))


def test_overlaps_are_refused(handle):
    """Outputs and the workspace are apart from the inputs and from each other; neighbours may touch."""
    rows, H, I, G = 32, 128, 64, 2
    p = _problem([20, 12], H, I)
    size = moe.grouped_gemm_backward_workspace_size(rows, H, I, num_groups=G)
    two = torch.empty((2 * rows, H), dtype=BF, device="cuda")
    two[:rows] = p["a"]
    a, wdn = two[:rows], G * H * I
    weights = torch.empty((2 * wdn,), dtype=BF, device="cuda")
    wg, dg = weights[:wdn].view(G, I, H), weights[wdn:].view(G, I, H)
    wg.copy_(p["wg"])
    ws = torch.empty(2 * size, dtype=torch.uint8, device="cuda")

    def call(**kw):
        d = dict(a=a, dy=p["dy"], offsets=p["offsets"], wg=wg, wu=p["wu"], wd=p["wd"], da=two[rows:], dg=dg,
                 du=torch.empty_like(wg), dd=torch.empty_like(p["wd"]), ws=ws[:size])
        d.update(kw)
        moe.grouped_swiglu_backward(handle, d["a"], d["dy"], d["offsets"], d["wg"], d["wu"], d["wd"], d["da"], d["dg"],
                                    d["du"], d["dd"], d["ws"], num_groups=G, H=H, I=I)
        return d

    o = call()
    _against_formulas(p, dict(o, da=o["da"]))
    inside = ws[:rows * H * 2].view(BF).view(rows, H)
    for kw in (dict(da=a), dict(da=p["dy"]), dict(da=two[rows // 2:rows // 2 + rows]), dict(da=two[rows - 1:2 * rows - 1]),
               dict(dg=wg), dict(dg=weights[64:64 + wdn].view(G, I, H)), dict(du=p["wu"]), dict(dd=p["wd"]), dict(du=dg),
               dict(dd=dg.view(G, H, I)), dict(da=dg.view(-1)[:rows * H].view(rows, H)), dict(da=inside), dict(a=inside),
               dict(dy=inside), dict(offsets=ws[256:268].view(torch.int32))):
        with pytest.raises(moe.MoEError) as e:
            call(**kw)
        assert e.value.status == moe.MOE_ERR_INVALID_ARG, list(kw)
    call(wu=wg)  # inputs may be one tensor
    assert handle.device_status() == 0


@pytest.mark.parametrize("G,H,I", [(64, 1024, 768), (220, 512, 320), (220, 1024, 768)])
def test_strips_of_several_tiles(handle, G, H, I):
    """Many groups: strips of two, three and four tiles that share their A columns, groups longer than the ring beside
    them, with six stages and with five. Every group's results are, bit for bit, those of a call with few groups, whose
    strips are single tiles; then the same where rows past a group's end have to be cleared."""
    g = torch.Generator().manual_seed(G + H)
    counts = torch.randint(0, 70, (G,), generator=g).tolist()
    counts[3], counts[10], counts[20], counts[30], counts[40], counts[G - 1] = 0, 401, 384, 385, 320, 333
    p = _problem(counts, H, I, lead=2, trail=9, seed=G)
    clean = _run(handle, p)
    for e in range(0, G, 8):
        n = min(8, G - e)
        b, end = p["off"][e], p["off"][e + n]
        part = dict(p, off=[o - b for o in p["off"][e:e + n + 1]], a=p["a"][b:end].contiguous(), dy=p["dy"][b:end].contiguous(),
                    offsets=p["offsets"][e:e + n + 1] - b, wg=p["wg"][e:e + n].contiguous(), wu=p["wu"][e:e + n].contiguous(),
                    wd=p["wd"][e:e + n].contiguous(), G=n, rows=end - b)
        few = _run(handle, part)
        assert torch.equal(few["da"], clean["da"][b:end])
        assert all(torch.equal(few[k], clean[k][e:e + n]) for k in ("dg", "du", "dd")), e
    for where in ("outside", "inside"):
        q = dict(p, a=p["a"].clone(), dy=p["dy"].clone())
        q["dy"][p["off"][-1]:] = float("nan")
        hit = []
        if where == "inside":
            hit = [11, 21, 31]
            for e in hit:
                q["dy"][p["off"][e]:p["off"][e + 1]] = float("nan")
                q["a"][p["off"][e]:p["off"][e + 1]] = float("inf")
            assert all(counts[e] for e in hit)
        o = _run(handle, q)
        for e in range(G):
            if e not in hit:
                assert torch.equal(o["da"][p["off"][e]:p["off"][e + 1]], clean["da"][p["off"][e]:p["off"][e + 1]])
                assert all(torch.equal(o[k][e], clean[k][e]) for k in ("dg", "du", "dd")), (where, e)
        assert all(o["dd"][e].isnan().any() for e in hit)
