"""moe_combine_backward, moe_route_backward and moe_permute_backward against the formulas in 64 bits.

Tolerances (u = 2^-24, bf16's unit roundoff 2^-8):
  dy_perm  one product of two numbers, rounded to fp32 and then to bf16: 1.01 * 2^-8 of it.
  dtopk_w  a sum of H fp32 products: (H/256 + 64) u of the absolute sum.
  dlogits  K terms of differences of dtopk_w's values, sigmoids good to 4 u each: (K + 32) u of the absolute sum,
           on the kernel's own dtopk_w.
  dx       a sum of K + 1 bf16 numbers in fp32, rounded once: 1.01 * 2^-8 of it and (K + 1) u of the absolute sum.
"""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load(build_if_missing=True)
    return moe.Handle(0)


def _problem(handle, T, H, E, K, norm, seed=0, drop=0, skew=0.0):
    """Routing and permutation by the library itself, on random logits; `drop` pairs get an id out of range."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cfg = moe.make_config(T, H, E, K, 64, 0, 2.826, norm)
    logits = torch.randn((T, E), device="cuda", generator=g) * 2
    if skew:
        logits += torch.randn((1, E), device="cuda", generator=g) * skew
    idx = torch.empty((T, K), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, K), device="cuda")
    moe.route(handle, cfg, logits, idx, tw)
    sent = idx.clone()
    if drop:
        sent.view(-1)[torch.randperm(T * K, device="cuda", generator=g)[:drop]] = E + 5
    counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    perm, f2p = (torch.empty(max(T * K, 1), dtype=torch.int32, device="cuda") for _ in range(2))
    xp = torch.empty((T * K, H), dtype=BF, device="cuda")
    ws = torch.empty(moe.permute_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    x = torch.randn((T, H), device="cuda", generator=g).to(BF)
    moe.permute(handle, cfg, x, sent, counts, offsets, perm, f2p, xp, ws)
    if drop:
        assert handle.device_status() != 0  # the permutation reports the dropped pairs
    return cfg, g, logits, idx, tw, f2p[:T * K], x, xp


CASES = [  # T, H, E, K, route_norm, dropped pairs
    (1, 64, 1, 1, False, 0), (1, 4096, 192, 8, True, 0), (2, 64, 8, 2, True, 1), (7, 192, 33, 5, False, 3),
    (61, 4096, 192, 8, True, 0), (64, 1088, 64, 32, True, 9), (33, 320, 256, 9, False, 0), (129, 512, 1024, 17, True, 5),
    (301, 2048, 40, 8, True, 0), (1000, 128, 8, 8, True, 100), (40, 8192, 16, 3, True, 0), (3, 16448, 16, 4, True, 2),
]


@pytest.mark.parametrize("T,H,E,K,norm,drop", CASES)
def test_against_formulas(handle, T, H, E, K, norm, drop):
    cfg, g, logits, idx, tw, f2p, _, _ = _problem(handle, T, H, E, K, norm, drop=drop)
    TK, p = T * K, f2p.long().view(T, K)
    live = p >= 0
    assert int((~live).sum()) == drop
    rows = p.clamp(min=0)
    y = torch.randn((TK, H), device="cuda", generator=g)
    dout = (torch.randn((T, H), device="cuda", generator=g) * 0.02).to(BF)
    sentinel = torch.full((TK, H), 7.0, dtype=BF, device="cuda")
    dy, dtw = sentinel.clone(), torch.full((T, K), 9.0, device="cuda")
    dl = torch.full((T, E), 9.0, device="cuda")
    moe.combine_backward(handle, cfg, dout, y, tw, f2p, dy, dtw, topk_idx=idx, logits=logits, dlogits=dl)
    d64 = dout.double()
    terms = y.double()[rows] * d64[:, None, :]
    want, size = terms.sum(2) * live, terms.abs().sum(2)
    assert ((dtw.double() - want).abs() <= (H / 256 + 64) * U * size).all()
    assert (dtw[~live] == 0).all()
    want_dy = sentinel.double()
    want_dy[rows[live]] = (tw.double()[:, :, None] * d64[:, None, :])[live]
    assert ((dy.double() - want_dy).abs() <= 1.01 * B * want_dy.abs()).all()
    hit = torch.zeros(TK, dtype=torch.bool, device="cuda")
    hit[rows[live]] = True
    assert (dy[~hit] == 7.0).all()  # rows of dropped pairs are left alone
    # routing: the formula on the kernel's own dtopk_w
    sg = torch.sigmoid(torch.gather(logits, 1, idx.long()).double())
    dw = dtw.double()
    if norm:
        S = sg.sum(1, keepdim=True)
        diff = dw[:, :, None] - dw[:, None, :]
        inner, mag = (sg[:, None, :] * diff).sum(2) / S ** 2, (sg[:, None, :] * diff.abs()).sum(2) / S ** 2
    else:
        inner, mag = dw, dw.abs()
    c = 2.826 * sg * (1 - sg)
    want_l, size_l = (torch.zeros((T, E), dtype=torch.float64, device="cuda") for _ in range(2))
    want_l.scatter_(1, idx.long(), c * inner)
    size_l.scatter_(1, idx.long(), c * mag)
    assert ((dl.double() - want_l).abs() <= (K + 32) * U * size_l).all()
    if K == 1 and norm:
        assert (dl == 0).all()
    # the same without the routing, and the routing alone
    dy2, dtw2, dl2 = sentinel.clone(), torch.empty_like(dtw), torch.empty_like(dl)
    moe.combine_backward(handle, cfg, dout, y, tw, f2p, dy2, dtw2)
    moe.route_backward(handle, cfg, logits, idx, dtw2, dl2)
    assert torch.equal(dy2, dy) and torch.equal(dtw2, dtw) and torch.equal(dl2, dl)
    # permutation
    dxp = (torch.randn((TK, H), device="cuda", generator=g) * 0.02).to(BF)
    add = (torch.randn((T, H), device="cuda", generator=g) * 0.02).to(BF)
    for a in (None, add):
        dx = torch.empty((T, H), dtype=BF, device="cuda")
        moe.permute_backward(handle, cfg, dxp, f2p, dx, dx_add=a)
        parts = dxp.double()[rows] * live[:, :, None]
        want = parts.sum(1) + (a.double() if a is not None else 0)
        size = parts.abs().sum(1) + (a.double().abs() if a is not None else 0)
        assert ((dx.double() - want).abs() <= 1.01 * B * want.abs() + (K + 1) * U * size).all()
    inplace = add.clone()
    moe.permute_backward(handle, cfg, dxp, f2p, inplace, dx_add=inplace)
    assert torch.equal(inplace, dx)
    assert handle.device_status() == 0


def test_a_nan_stays_with_its_token(handle):
    cfg, g, logits, idx, tw, f2p, _, _ = _problem(handle, 50, 256, 16, 4, True)
    y, dout = torch.randn((200, 256), device="cuda", generator=g), torch.randn((50, 256), device="cuda", generator=g).to(BF)
    bufs = lambda: (torch.empty((200, 256), dtype=BF, device="cuda"), torch.empty((50, 4), device="cuda"),  # noqa: E731
                    torch.empty((50, 16), device="cuda"))
    a, b = bufs(), bufs()
    moe.combine_backward(handle, cfg, dout, y, tw, f2p, a[0], a[1], topk_idx=idx, logits=logits, dlogits=a[2])
    p = f2p.view(50, 4).long()
    y[p[20, 1], 3] = float("nan")
    moe.combine_backward(handle, cfg, dout, y, tw, f2p, b[0], b[1], topk_idx=idx, logits=logits, dlogits=b[2])
    assert torch.equal(a[0], b[0])
    others = torch.arange(50, device="cuda") != 20
    assert torch.equal(a[1][others], b[1][others]) and torch.equal(a[2][others], b[2][others])
    assert b[1][20, 1].isnan() and not b[1][20, 0].isnan()


@pytest.mark.parametrize("norm", [True, False])
def test_route_backward_against_differences(handle, norm):
    """<dlogits, v> against central differences, in 64 bits, of sum(c * w(logits)) with the chosen experts fixed."""
    T, E, K = 20, 24, 6
    cfg, g, logits, idx, _, _, _, _ = _problem(handle, T, 64, E, K, norm)
    c = torch.randn((T, K), device="cuda", generator=g)
    dl = torch.empty((T, E), device="cuda")
    moe.route_backward(handle, cfg, logits, idx, c, dl)

    def loss(l):
        s = torch.sigmoid(torch.gather(l, 1, idx.long()))
        return (c.double() * 2.826 * (s / s.sum(1, keepdim=True) if norm else s)).sum()

    v, t = torch.randn((T, E), device="cuda", generator=g).double(), 1e-5
    diff = (loss(logits.double() + t * v) - loss(logits.double() - t * v)) / (2 * t)
    # fp32 of the gradient ((K + 32) u of its terms, at most a few times it here) and the t^2 of the differences
    assert ((dl.double() * v).sum() - diff).abs() <= 1e-5 * (dl.double() * v).abs().sum()


def test_combine_backward_against_differences(handle):
    """combine is linear in y, w and shared: <dy, v> and <dw, v> are differences of the formula itself."""
    T, H, E, K = 9, 128, 12, 3
    cfg, g, logits, idx, tw, f2p, x, xp = _problem(handle, T, H, E, K, True)
    y, dout = torch.randn((T * K, H), device="cuda", generator=g), torch.randn((T, H), device="cuda", generator=g).to(BF)
    dy, dtw = torch.empty((T * K, H), dtype=BF, device="cuda"), torch.empty((T, K), device="cuda")
    moe.combine_backward(handle, cfg, dout, y, tw, f2p, dy, dtw)
    p = f2p.view(T, K).long()
    loss = lambda yy, ww: (dout.double() * (ww[:, :, None] * yy[p]).sum(1)).sum()  # noqa: E731
    vy, vw = torch.randn((T * K, H), device="cuda", generator=g).double(), torch.randn((T, K), device="cuda", generator=g).double()
    dif = loss(y.double() + vy, tw.double()) - loss(y.double(), tw.double())
    assert ((dy.double() * vy).sum() - dif).abs() <= 1.02 * B * (dy.double() * vy).abs().sum()
    dif = loss(y.double(), tw.double() + vw) - loss(y.double(), tw.double())
    assert ((dtw.double() * vw).sum() - dif).abs() <= 65 * U * (dout.double().abs()[:, None, :] * y.double()[p].abs() *
                                                               vw.abs()[:, :, None]).sum()
    # permute: <x_perm, v> = <x, permute_backward(v)>
    v = torch.randn((T * K, H), device="cuda", generator=g).to(BF)
    dx = torch.empty((T, H), dtype=BF, device="cuda")
    moe.permute_backward(handle, cfg, v, f2p, dx)
    assert ((xp.double() * v.double()).sum() - (x.double() * dx.double()).sum()).abs() <= \
        1.01 * B * (x.double() * dx.double()).abs().sum()


def test_no_tokens_bad_indices_and_refusals(handle):
    cfg0 = moe.make_config(0, 64, 8, 2, 64, 0, 1.0)
    e = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    moe.combine_backward(handle, cfg0, e(0, 64, dt=BF), e(0, 64), e(0, 2), e(0, dt=i32), e(0, 64, dt=BF), e(0, 2))
    moe.permute_backward(handle, cfg0, e(0, 64, dt=BF), e(0, dt=i32), e(0, 64, dt=BF))
    cfg, g, logits, idx, tw, f2p, _, _ = _problem(handle, 6, 64, 8, 2, True)
    y, dout = torch.randn((12, 64), device="cuda", generator=g), torch.randn((6, 64), device="cuda", generator=g).to(BF)
    dy, dtw, dl = torch.zeros((12, 64), dtype=BF, device="cuda"), e(6, 2), e(6, 8)
    bad = f2p.clone()
    bad[3] = 12
    moe.combine_backward(handle, cfg, dout, y, tw, bad, dy, dtw)
    assert dtw[1, 1] == 0 and handle.device_status() == 17  # MOE_DEV_BAD_PERM_INDEX, and the word is cleared
    wrong = idx.clone()
    wrong[2, 0] = 8
    moe.combine_backward(handle, cfg, dout, y, tw, f2p, dy, dtw, topk_idx=wrong, logits=logits, dlogits=dl)
    assert handle.device_status() == 16  # MOE_DEV_BAD_EXPERT_ID
    assert dl[2].isfinite().all() and int((dl[2] != 0).sum()) <= 1
    args = (handle, cfg, dout, y, tw, f2p, dy, dtw)
    for kw in (dict(logits=logits), dict(topk_idx=idx, logits=logits), dict(topk_idx=idx, logits=logits, dlogits=logits)):
        with pytest.raises(moe.MoEError):
            moe.combine_backward(*args, **kw)
    for i, t in ((2, dout.float()), (3, y.bfloat16()), (5, f2p.long()), (6, dy[:6]), (7, None), (3, y.t().contiguous().t())):
        a = list(args)
        a[i] = t
        with pytest.raises(moe.MoEError):
            moe.combine_backward(*a)
    with pytest.raises(moe.MoEError):
        moe.permute_backward(handle, cfg, dy, f2p, dout, dx_add=dout.float())
    with pytest.raises(moe.MoEError):
        moe.route_backward(handle, cfg, logits, idx, dtw, logits)
    assert handle.device_status() == 0


@pytest.mark.parametrize("lo,hi,std", [(-88.6, -86.0, 1.0), (-88.6, -88.0, 300.0), (-60.0, -40.0, 1.0), (20.0, 90.0, 1.0)])
def test_routing_weights_of_far_logits(handle, lo, hi, std):
    """Weights divided by their sum stay of order one however small the sigmoids are, and so does their gradient.
    Down to 1e-39, where fp32 has 2^-150 of absolute rounding left, a sigmoid is good to 4 u, so a weight to (K + 18) u
    and the gradient, two weights and a sum of K terms, to (2 K + 48) u of its absolute sum; 1 - sigma is good to 4 u or, below
    fp32's normal numbers, to 2^-126."""
    T, H, E, K = 70, 64, 24, 6
    g = torch.Generator(device="cuda").manual_seed(11)
    cfg = moe.make_config(T, H, E, K, 64, 0, 2.826, True)
    logits = torch.rand((T, E), device="cuda", generator=g) * (hi - lo) + lo
    idx, tw = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    moe.route(handle, cfg, logits, idx, tw)
    assert tw.isfinite().all()
    dw, dl = torch.randn((T, K), device="cuda", generator=g) * std, torch.empty((T, E), device="cuda")
    moe.route_backward(handle, cfg, logits, idx, dw, dl)
    l = torch.gather(logits, 1, idx.long()).double()
    sg, om = torch.sigmoid(l), torch.sigmoid(-l)
    r = sg / sg.sum(1, keepdim=True)
    diff = dw.double()[:, :, None] - dw.double()[:, None, :]
    want = 2.826 * r * om * (r[:, None, :] * diff).sum(2)
    size = 2.826 * r * om * (r[:, None, :] * diff.abs()).sum(2)
    got = torch.gather(dl, 1, idx.long()).double()
    assert ((got - want).abs() <= ((2 * K + 48) * U + 2.0 ** -126 / om) * size + 2.0 ** -149).all()
    rest = dl.clone().scatter_(1, idx.long(), 0.0)
    assert (rest == 0).all()
    # with the combine's gradient in front: y such that dtopk_w is dw, exactly
    f2p = torch.arange(T * K, dtype=torch.int32, device="cuda")
    y, dout = torch.zeros((T * K, H), device="cuda"), torch.zeros((T, H), dtype=BF, device="cuda")
    y[:, 3], dout[:, 3] = dw.view(-1), 1.0
    dl2, dtw, dy = torch.empty_like(dl), torch.empty_like(dw), torch.empty((T * K, H), dtype=BF, device="cuda")
    moe.combine_backward(handle, cfg, dout, y, tw, f2p, dy, dtw, topk_idx=idx, logits=logits, dlogits=dl2)
    assert torch.equal(dtw, dw) and torch.equal(dl2, dl)


@pytest.mark.parametrize("T,H,E,K,norm,drop", [
    (700, 4096, 192, 8, True, 40), (1021, 1088, 64, 5, False, 7), (2600, 4096, 192, 8, True, 0),  # passes, waves of blocks
    (5000, 512, 64, 4, True, 3), (900, 2112, 40, 20, True, 11)])
def test_batches(handle, T, H, E, K, norm, drop):
    test_against_formulas(handle, T, H, E, K, norm, drop)
