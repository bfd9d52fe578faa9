"""moe_add_rmsnorm and moe_add_rmsnorm_backward against the formulas in 64 bits.

Tolerances (u = 2^-24, the fp32 unit roundoff; bf16's is 2^-8):
  h_out   the correctly rounded fp32 sum: bit-equal.
  rstd    at most H/256 + 48 roundings of a sum of squares, halved by the root,
          plus the division and the root: (H/256 + 48) u.
  out     one rounding to bf16 of n, whose own error is far below it: 1.02 * 2^-8 |n|.
  MXFP8   the codes are those of n perturbed by at most 1e-5 (ties and powers of
          two may fall either way inside that).
  dh      one rounding to bf16 (or none, fp32 stream) on top of fp32 arithmetic
          whose terms are bounded by their absolute sum: (H/256 + 64) u of it.
  dweight a sum of `rows` fp32 terms: (rows + 64) u of its absolute sum.
"""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-5


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load(build_if_missing=True)
    return moe.Handle(0)


def _randn(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def _e4m3_codes(v):
    """E4M3 codes of fp64 values, nearest even, saturating."""
    return v.clamp(-448, 448).to(F32).to(torch.float8_e4m3fn).view(torch.uint8)


def _mx(n):
    b = n.reshape(-1, 32)
    amax = b.abs().amax(1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent.long() - 9, torch.full_like(amax, -127).long()).clamp(-127, 127)
    codes = _e4m3_codes(b * torch.exp2(-e.double())[:, None])
    return codes.reshape(n.shape), torch.where(amax > 0, e + 127, torch.zeros_like(e)).to(torch.uint8).reshape(
        n.shape[0], -1)


def _forward64(x, r, w, eps=EPS):
    s = x.double() + (r.double() if r is not None else 0.0)
    rstd = 1.0 / torch.sqrt((s * s).mean(1) + eps)
    return s, rstd, s * rstd[:, None] * w.double()


def _run(handle, x, r, w, rt, mx=False, eps=EPS, with_h=True):
    rows, H = x.shape
    o = dict(h=torch.empty((rows, H), dtype=rt, device="cuda") if with_h else None,
             out=torch.empty((rows, H), dtype=BF, device="cuda"),
             rstd=torch.empty(rows, dtype=F32, device="cuda"), q=None, s=None)
    if mx:
        o["q"] = torch.empty((rows, H), dtype=torch.uint8, device="cuda")
        o["s"] = torch.empty((rows, H // 32), dtype=torch.uint8, device="cuda")
    for t in o.values():
        if t is not None:
            t.view(torch.uint8).fill_(0xA5)
    moe.add_rmsnorm(handle, x, w, eps, residual=r, h_out=o["h"], out=o["out"], q=o["q"], q_scale=o["s"], rstd=o["rstd"])
    return o


CASES = [  # rows, H, residual, MXFP8
    (1, 8, "bf16", False), (1, 1, "f32", False), (3, 250, "bf16", False), (5, 1001, "f32", False),
    (2, 32, None, True), (9, 96, "bf16", True), (333, 256, "f32", True), (17, 264, "bf16", False),
    (8, 512, "bf16", True), (65, 992, "f32", True), (7, 1024, "bf16", True), (7, 1032, "f32", False),
    (1, 4096, "bf16", True), (64, 4096, "bf16", True), (61, 4096, "f32", True), (500, 4096, None, True),
    (5, 8192, "bf16", True), (3, 8200, "f32", False), (4, 16384, "bf16", True), (2, 16384, "f32", True),
    (2, 16383, "bf16", False), (40000, 64, "bf16", True),
]


@pytest.mark.parametrize("rows,H,res,mx", CASES)
def test_forward(handle, rows, H, res, mx):
    rt = F32 if res == "f32" else BF
    x, w = _randn((rows, H), BF, 1), (1 + 0.2 * _randn((H,), F32, 2)).to(BF)
    r = _randn((rows, H), rt, 3, 3.0) if res else None
    o = _run(handle, x, r, w, rt, mx)
    s, rstd, n = _forward64(x, r, w)
    want_h = x.float() + (r.float() if r is not None else 0.0)
    assert torch.equal(o["h"], want_h.to(rt))
    assert ((o["rstd"].double() - rstd).abs() <= (H / 256 + 48) * U * rstd).all()
    assert ((o["out"].double() - n).abs() <= 1.02 * B * n.abs()).all()
    if mx:
        lo, hi = _mx(n * (1 - 1e-5)), _mx(n * (1 + 1e-5))
        assert ((o["s"] == lo[1]) | (o["s"] == hi[1])).all()
        same = (lo[1] == hi[1]).repeat_interleave(32, 1)  # blocks whose scale is not in question
        assert ((o["q"] == lo[0]) | (o["q"] == hi[0]) | ~same).all()
        assert same.float().mean() > 0.99 or rows * H < 3200
    assert handle.device_status() == 0


def test_zero_inf_and_nan_rows_stay_in_their_rows(handle):
    rows, H = 6, 4096
    x, w = _randn((rows, H), BF, 1), torch.ones(H, dtype=BF, device="cuda")
    clean = _run(handle, x, None, w, BF, True)
    x[1] = 0
    x[3, 17] = float("nan")
    x[4, 5] = float("inf")
    x[2, 32:64] = 0  # one empty block
    o = _run(handle, x, None, w, BF, True)
    assert (o["out"][1] == 0).all() and (o["q"][1] == 0).all() and (o["s"][1] == 0).all()
    assert abs(o["rstd"][1].item() - EPS ** -0.5) < 1e-4 * EPS ** -0.5
    assert o["out"][3].isnan().all() and ((o["q"][3] & 0x7F) == 0x7F).all() and (o["s"][3] == 247).all()
    assert o["out"][4, 5].isnan() and (o["out"][4, :5] == 0).all()  # inf * 0 and finite * 0
    assert (o["q"][2, 32:64] == 0).all() and o["s"][2, 1] == 0
    for k in ("out", "q", "s", "rstd", "h"):
        for row in (0, 5):
            assert torch.equal(o[k][row], clean[k][row]), k


@pytest.mark.parametrize("H", [64, 250, 4096])
def test_in_place_no_rows_and_another_stream(handle, H):
    x, r, w = _randn((33, H), BF, 1), _randn((33, H), BF, 2), _randn((H,), BF, 3)
    want = _run(handle, x, r, w, BF)
    x2, r2 = x.clone(), r.clone()
    moe.add_rmsnorm(handle, x2, w, EPS, residual=r2, h_out=r2, out=x2)
    assert torch.equal(x2, want["out"]) and torch.equal(r2, want["h"])
    side = torch.cuda.Stream()
    out = torch.empty_like(x)
    side.wait_stream(torch.cuda.current_stream())
    moe.add_rmsnorm(handle, x, w, EPS, residual=r, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want["out"])
    e = torch.empty((0, H), dtype=BF, device="cuda")
    moe.add_rmsnorm(handle, e, w, EPS, out=e)
    dw = torch.full((H,), 3.0, device="cuda")
    ws = torch.empty(moe.add_rmsnorm_backward_workspace_size(0, H), dtype=torch.uint8, device="cuda")
    moe.add_rmsnorm_backward(handle, e, e, w, torch.empty(0, device="cuda"), e, ws, dweight=dw)
    assert (dw == 0).all()


def test_mx_output_is_the_layers_quantisation(handle):
    """With weight 1 and bf16-exact n (rows of +-1: rstd = 1 up to eps) the codes are moe_quantize_mxfp8's."""
    x = torch.where(_randn((64, 512), F32, 4) > 0, 2.0, -2.0).to(BF)
    w = torch.ones(512, dtype=BF, device="cuda")
    o = _run(handle, x, None, w, BF, True, eps=0.0)
    q, s = moe.quantize_mx(handle, o["out"])
    assert torch.equal(q, o["q"]) and torch.equal(s, o["s"])


def _backward64(dout, h, w, rstd, dh_in):
    xh, g = h.double() * rstd.double()[:, None], dout.double() * w.double()
    m = (g * xh).mean(1, keepdim=True)
    r = rstd.double()[:, None]
    dh = r * (g - xh * m) + (dh_in.double() if dh_in is not None else 0.0)
    size = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + (dh_in.double().abs() if dh_in is not None else 0)
    return dh, size, (dout.double() * xh).sum(0), (dout.double() * xh).abs().sum(0)


BWD = [(1, 8, "bf16", True), (1, 1, "f32", False), (5, 250, "bf16", True), (700, 1001, "f32", True),
       (333, 256, "f32", True), (9, 512, "bf16", False), (2600, 1024, "bf16", True), (70, 1032, "f32", True),
       (1, 4096, "bf16", True), (1000, 4096, "bf16", True), (305, 4096, "f32", True), (304, 8192, "bf16", False),
       (7, 8200, "f32", True), (310, 16384, "bf16", True), (3, 16384, "f32", True), (2, 16383, "bf16", True)]


@pytest.mark.parametrize("rows,H,res,has_in", BWD)
def test_backward(handle, rows, H, res, has_in):
    rt = F32 if res == "f32" else BF
    h, dout = _randn((rows, H), rt, 5, 3.0), _randn((rows, H), BF, 6, 0.02)
    w = (1 + 0.2 * _randn((H,), F32, 7)).to(BF)
    dh_in = _randn((rows, H), rt, 8, 0.02) if has_in else None
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dh, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    dx = torch.empty((rows, H), dtype=BF, device="cuda")
    ws = torch.empty(moe.add_rmsnorm_backward_workspace_size(rows, H), dtype=torch.uint8, device="cuda").fill_(0xFF)
    moe.add_rmsnorm_backward(handle, dout, h, w, rstd, dh, ws, dh_in=dh_in, dx=dx, dweight=dw)
    want, size, want_w, size_w = _backward64(dout, h, w, rstd, dh_in)
    fp = (H / 256 + 64) * U * size
    assert ((dh.double() - want).abs() <= fp + (1.02 * B * want.abs() if rt == BF else 0)).all()
    assert ((dx.double() - want).abs() <= fp + 1.02 * B * want.abs()).all()
    assert ((dw.double() - want_w).abs() <= (rows + 64) * U * size_w + 1e-30).all()
    again_h, again_w = torch.empty_like(h), torch.empty_like(dw)
    moe.add_rmsnorm_backward(handle, dout, h, w, rstd, again_h, ws, dh_in=dh_in, dweight=again_w)
    assert torch.equal(again_h, dh) and torch.equal(again_w, dw)
    if has_in:  # dh over dh_in, dx over dout
        d2, i2 = dout.clone(), dh_in.clone()
        moe.add_rmsnorm_backward(handle, d2, h, w, rstd, i2, None, dh_in=i2, dx=d2)
        assert torch.equal(i2, dh) and torch.equal(d2, dx)


@pytest.mark.parametrize("H", [96, 1000, 2048])
def test_backward_against_differences(handle, H):
    """<dh, v> and <dweight, u> against central differences, in 64 bits, of sum(c * n(h, w))."""
    rows = 12
    h, w, c = _randn((rows, H), F32, 1, 2.0), (1 + 0.2 * _randn((H,), F32, 2)).to(BF), _randn((rows, H), BF, 3)
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    dh, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    ws = torch.empty(moe.add_rmsnorm_backward_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    moe.add_rmsnorm_backward(handle, c, h, w, rstd, dh, ws, dweight=dw)
    loss = lambda hh, ww: (c.double() * hh * (1 / torch.sqrt((hh * hh).mean(1, keepdim=True) + EPS)) * ww).sum()  # noqa: E731
    v, t = _randn((rows, H), F64, 4), 1e-5
    diff = (loss(h.double() + t * v, w.double()) - loss(h.double() - t * v, w.double())) / (2 * t)
    got = (dh.double() * v).sum()
    # The differences are good to t^2; the gradient to (H/256 + 64 + rstd's 8) u of its terms.
    assert (got - diff).abs() <= 200 * U * (dh.double() * v).abs().sum() + 1e-6 * (dh.double() * v).norm()
    v = _randn((H,), F64, 5)
    diff = (loss(h.double(), w.double() + t * v) - loss(h.double(), w.double() - t * v)) / (2 * t)
    assert ((dw.double() * v).sum() - diff).abs() <= 200 * U * (dw.double() * v).abs().sum() + 1e-6 * (dw.double() * v).norm()


def test_refusals(handle):
    x, w = _randn((4, 64), BF, 1), _randn((64,), BF, 2)
    out = torch.empty_like(x)
    q, s = torch.empty((4, 64), dtype=torch.uint8, device="cuda"), torch.empty((4, 2), dtype=torch.uint8, device="cuda")
    bad = [dict(),                                                   # neither out nor q
           dict(out=out, q=q), dict(out=out, q_scale=s),             # codes without scales
           dict(out=out.float()), dict(out=out[:2]),                 # type, size
           dict(out=torch.empty((64, 4), dtype=BF, device="cuda").t()),  # layout
           dict(out=torch.empty((4, 64), dtype=BF)),                 # device
           dict(out=out, residual=x.half()), dict(out=out, residual=x, h_out=x.float())]
    for kw in bad:
        with pytest.raises(moe.MoEError):
            moe.add_rmsnorm(handle, x, w, EPS, **kw)
    for eps in (float("nan"), float("inf"), -1.0):
        with pytest.raises(moe.MoEError):
            moe.add_rmsnorm(handle, x, w, eps, out=out)
    with pytest.raises(moe.MoEError):  # MXFP8 needs whole blocks of 32
        moe.add_rmsnorm(handle, x[:, :40].contiguous(), w[:40].contiguous(), EPS,
                        q=torch.empty((4, 40), dtype=torch.uint8, device="cuda"),
                        q_scale=torch.empty(5, dtype=torch.uint8, device="cuda"))
    rstd, dw = torch.ones(4, device="cuda"), torch.empty(64, device="cuda")
    with pytest.raises(moe.MoEError) as e:  # dweight without a workspace
        moe.add_rmsnorm_backward(handle, x, x, w, rstd, out, None, dweight=dw)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoEError) as e:
        moe.add_rmsnorm_backward(handle, x, x, w, rstd, out, torch.empty(16, dtype=torch.uint8, device="cuda"), dweight=dw)
    assert e.value.status == moe.MOE_ERR_WORKSPACE
    assert handle.device_status() == 0


LONG = [  # rows, H, residual: every group walks its ring at least twice over
    (4000, 4096, "f32"), (6000, 1024, "f32"), (3000, 8192, "f32"), (1500, 8200, "f32"), (1500, 16384, "f32"),
    (30000, 256, "f32"), (30000, 256, "bf16"), (30000, 512, "bf16"), (8000, 4096, "bf16"), (1500, 9216, "bf16"),
    (1500, 16384, "bf16"), (5003, 1000, "bf16"),
]


@pytest.mark.parametrize("has_in", [True, False])
@pytest.mark.parametrize("rows,H,res", LONG)
def test_backward_over_many_rows(handle, rows, H, res, has_in):
    test_backward(handle, rows, H, res, has_in)
    rt = F32 if res == "f32" else BF
    h, dout = _randn((rows, H), rt, 5, 3.0), _randn((rows, H), BF, 6, 0.02)
    w = (1 + 0.2 * _randn((H,), F32, 7)).to(BF)
    dh_in = _randn((rows, H), rt, 8, 0.02) if has_in else None
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    ws = torch.empty(moe.add_rmsnorm_backward_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    dh, dx, dw = torch.empty_like(h), torch.empty_like(dout), torch.empty(H, device="cuda")
    moe.add_rmsnorm_backward(handle, dout, h, w, rstd, dh, ws, dh_in=dh_in, dx=dx, dweight=dw)
    h2, d2, dw2 = h.clone(), dout.clone(), torch.empty_like(dw)  # dh over h, dx over dout
    moe.add_rmsnorm_backward(handle, d2, h2, w, rstd, h2, ws, dh_in=dh_in, dx=d2, dweight=dw2)
    assert torch.equal(h2, dh) and torch.equal(d2, dx) and torch.equal(dw2, dw)
