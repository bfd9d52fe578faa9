"""E4M3 with one fp32 scale per block of 128 at its edges: scales so small that a quotient's remainder is subnormal, the
layer's answer under an option that only sizes its launches, and sums shared between thread blocks over many launches."""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe
import synth
from test_gpu_fp8 import quantize64
from test_gpu_fp8_layer import problem

pytestmark = pytest.mark.gpu

E4M3, F32, F64, U8 = torch.float8_e4m3fn, torch.float32, torch.float64, torch.uint8


@pytest.fixture(scope="module")
def handle():
    h = moe.Handle(0)
    yield h
    torch.cuda.synchronize()
    assert h.device_status() == 0
    h.close()


# ---------------------------------------------------------------- quotients
def near_borders(n, exponent, seed):
    """n blocks of 128 fp32 values whose scale is in [2^exponent, 2^(exponent + 1)): the largest, then values a step of
    fp32 around the scale times each border between two codes, and the codes that the rule asks for. The quotient rounded
    to fp32 is that of the 64-bit quotient, as 53 bits are at least twice 24 and two more."""
    g = torch.Generator().manual_seed(seed)
    every = torch.arange(0x7F, dtype=U8).view(E4M3).to(F64)  # 0 .. 448
    border = (every[1:] + every[:-1]) / 2
    amax = (448 * 2.0 ** exponent * (1 + torch.rand(n, generator=g, dtype=F64) * 0.999)).to(F32)
    s = (amax.to(F64) / 448).to(F32)
    b = border[torch.randint(0, border.numel(), (n, 128), generator=g)]
    v = (b * s.to(F64)[:, None]).to(F32)
    v = (v.view(torch.int32) + torch.randint(-1, 2, (n, 128), generator=g, dtype=torch.int32)).view(F32)
    v = v * torch.where(torch.rand((n, 128), generator=g) < 0.5, -1.0, 1.0)
    v[:, 0] = amax
    return v, s, codes_of(v, s[:, None])


def codes_of(v, s):
    return (v.to(F64) / s.to(F64)).to(F32).clamp(-448, 448).to(E4M3)


EXPONENTS = [-126, -125, -120, -116, -112, -104, -96, -81, -80, -79, -60, 0, 100]


@pytest.mark.parametrize("exponent", EXPONENTS)
def test_rows_and_columns_near_borders(handle, exponent):
    v, s, want = near_borders(2048, exponent, seed=exponent + 1000)
    x = v.reshape(256, 1024).cuda()
    q, sc = torch.empty(x.shape, dtype=U8, device="cuda"), torch.empty((256, 8), device="cuda")
    moe.quantize_fp8(handle, x, q, sc)
    assert torch.equal(sc.cpu().reshape(-1), s)
    assert torch.equal(q.cpu().view(E4M3).float().reshape(-1, 128), want.float())
    x = v[:1024].t().contiguous().cuda()  # a block per column
    q, sc = torch.empty((256, 1024), dtype=U8, device="cuda"), torch.empty((2, 1024), device="cuda")
    moe.quantize_fp8_columns(handle, x, None, q, sc, num_groups=1)
    assert torch.equal(sc[0].cpu(), s[:1024])
    assert torch.equal(q[:128].cpu().view(E4M3).float().t(), want[:1024].float())


@pytest.mark.parametrize("exponent", EXPONENTS)
def test_squares_near_borders(handle, exponent):
    """128 blocks of one scale: the first one's largest value, the others' values around its borders."""
    g = torch.Generator().manual_seed(exponent + 2000)
    v, s, _ = near_borders(1, exponent, seed=exponent + 3000)
    every = torch.arange(0x7F, dtype=U8).view(E4M3).to(F64)
    b = ((every[1:] + every[:-1]) / 2)[torch.randint(0, 126, (128, 128), generator=g)]
    x = (b * s.to(F64)).to(F32)
    x = (x.view(torch.int32) + torch.randint(-1, 2, (128, 128), generator=g, dtype=torch.int32)).view(F32)
    x[17, 5] = v[0, 0]
    q, sc = torch.empty((128, 128), dtype=U8, device="cuda"), torch.empty((1, 1), device="cuda")
    moe.quantize_fp8(handle, x.cuda(), q, sc, squares=True)
    assert float(sc) == float(s)
    assert torch.equal(q.cpu().view(E4M3).float(), codes_of(x, s).float())


def test_scales_of_all_sizes_side_by_side(handle):
    """Small and large scales, zeros and a NaN in neighbouring blocks, rows and columns."""
    parts = [near_borders(64, EXPONENTS[i % len(EXPONENTS)], seed=5000 + i) for i in range(2 * len(EXPONENTS))]
    v, s, want = (torch.cat([p[i].float() if i == 2 else p[i] for p in parts]) for i in range(3))
    order = torch.randperm(v.shape[0], generator=torch.Generator().manual_seed(7))
    v, s, want = v[order], s[order], want[order]
    v[5], s[5], want[5] = 0.0, 2.0 ** -126, 0.0
    n = v.shape[0]
    x = v.reshape(n // 8, 1024).cuda()
    q, sc = torch.empty(x.shape, dtype=U8, device="cuda"), torch.empty((n // 8, 8), device="cuda")
    moe.quantize_fp8(handle, x, q, sc)
    assert torch.equal(sc.cpu().reshape(-1), s) and torch.equal(q.cpu().view(E4M3).float().reshape(-1, 128), want)
    x = v.t().contiguous().cuda()
    x[3, 9] = float("nan")
    q, sc = torch.empty((256, n), dtype=U8, device="cuda"), torch.empty((2, n), device="cuda")
    moe.quantize_fp8_columns(handle, x, None, q, sc, num_groups=1)
    rest = torch.arange(n) != 9
    got = q[:128].cpu().view(E4M3).float().t()
    assert torch.equal(sc[0].cpu()[rest], s[rest]) and torch.equal(got[rest], want[rest])
    assert sc[0, 9].isnan() and got[9].isnan().all()


@pytest.mark.parametrize("exponent", [-125, -116, -100])
def test_bf16_small_scales(handle, exponent):
    g = torch.Generator().manual_seed(exponent + 4000)
    x = (448 * 2.0 ** exponent * torch.randn((512, 1024), generator=g, dtype=F64)).to(torch.bfloat16)
    amax = x.to(F64).abs().reshape(512, 8, 128).amax(2)
    s = (amax / 448).to(F32).clamp(min=2.0 ** -126)
    q, sc = torch.empty(x.shape, dtype=U8, device="cuda"), torch.empty((512, 8), device="cuda")
    moe.quantize_fp8(handle, x.cuda(), q, sc)
    assert torch.equal(sc.cpu(), s)
    want = codes_of(x.reshape(512, 8, 128), s[:, :, None]).reshape(512, 1024)
    assert torch.equal(q.cpu().view(E4M3).float(), want.float())


@pytest.mark.parametrize("rows, H, I", [(300, 256, 400), (7, 4096, 272), (33, 2560, 128)])
def test_gate_up_of_small_scales(handle, rows, H, I):
    """The up weights' scales times 2^-100: the same codes, and scales times 2^-100 (every step of it is exact)."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    code = lambda *s: (130.0 * torch.randn(s, device="cuda", generator=g)).clamp(-448, 448).to(E4M3).view(U8)  # noqa: E731
    scale = lambda std, *s: std * (0.5 + torch.rand(s, device="cuda", generator=g))  # noqa: E731
    nh, ni = -(-H // 128), -(-I // 128)
    a, sa, wg, wu = code(rows, H), scale(0.01, rows, nh), code(1, I, H), code(1, I, H)
    sg, su = scale(2e-4, 1, ni, nh), scale(2e-4, 1, ni, nh)
    got = []
    for k in (0, -100):
        q, s = torch.empty((rows, I), dtype=U8, device="cuda"), torch.empty((rows, ni), device="cuda")
        moe.grouped_gate_up_fp8(handle, a, sa, None, wg, sg, wu, su * 2.0 ** k, q, s, num_groups=1, H=H, I=I)
        got.append((q, s))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1] * 2.0 ** -100, got[1][1])
    assert (got[1][1] < 2.0 ** -80).all()


@pytest.mark.parametrize("form", ["rows", "squares", "columns"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, F32])
@pytest.mark.parametrize("R, C", [(301, 4112), (33, 2064), (1000, 1040), (2, 65536), (5, 65520)])
def test_wide_rows(handle, R, C, dtype, form):
    """More blocks per row than a thread block takes at a time, whole ones and not, up to the widest that products take."""
    x = torch.randn((R, C), device="cuda", generator=torch.Generator(device="cuda").manual_seed(R + C)).to(dtype)
    height, width = {"rows": (1, 128), "squares": (128, 128), "columns": (128, 1)}[form]
    want, sw = quantize64(x, height, width)
    P = moe.fp8_padded_rows(R) if form == "columns" else R
    q = torch.empty((P, C), dtype=U8, device="cuda")
    s = torch.empty((P // 128 if form == "columns" else sw.shape[0], sw.shape[1]), device="cuda")
    if form == "columns":
        moe.quantize_fp8_columns(handle, x, None, q, s, num_groups=1)
    else:
        moe.quantize_fp8(handle, x, q, s, squares=form == "squares")
    assert torch.equal(s[:sw.shape[0]], sw[:, :s.shape[1]]) and torch.equal(q[:R].view(E4M3).float(), want.view(E4M3).float())


# ---------------------------------------------------------------- the layer's option for the shared expert's SMs
@pytest.mark.parametrize("shape", [
    synth.MoEShape("fd", T=9, H=4096, E=3, K=1, I=128, I_shared=256, dtype="fp8"),
    synth.MoEShape("fe", T=33, H=2560, E=4, K=2, I=2560, I_shared=2560, dtype="fp8"),
    synth.MoEShape("ff", T=300, H=512, E=32, K=4, I=256, I_shared=256, dtype="fp8")], ids=lambda s: s.name)
def test_shared_sms_do_not_change_the_result(shape):
    """MOE_OPT_SHARED_SMS gives the same bits whatever it is, also where a product's reduction is shared out."""
    x, logits, w = problem(shape, 2)
    layer = moe.MoELayer(shape, w, device=0)
    out = layer(x, logits).clone()
    for k in (1, 4, 8, 40, 60, 1000):
        layer.handle.set_option(moe.MOE_OPT_SHARED_SMS, k)
        assert torch.equal(layer(x, logits), out), f"{k} SMs"
    assert layer.handle.device_status() == 0


# ---------------------------------------------------------------- parts of a reduction
@pytest.mark.parametrize("rows, N, K", [(7, 1536, 4096), (1, 256, 4080), (40, 512, 4096), (64, 2304, 2704)])
def test_parts_over_many_launches(handle, rows, N, K):
    """The sums that a cluster's thread blocks send each other, over launches back to back with inputs that alternate:
    each launch gives its own inputs' bits."""
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    nb = -(-K // 128)
    sets = []
    for _ in range(2):
        code = lambda *s: (130.0 * torch.randn(s, device="cuda", generator=g)).clamp(-448, 448).to(E4M3).view(U8)  # noqa: E731
        scale = lambda *s: 1e-3 * (0.5 + torch.rand(s, device="cuda", generator=g))  # noqa: E731
        sets.append((code(rows, K), scale(rows, nb), code(1, N, K), scale(1, -(-N // 128), nb)))
    outs = torch.zeros((200, rows, N), device="cuda")
    qs = torch.zeros((200, rows, N), dtype=U8, device="cuda")
    ss = [torch.zeros((rows, -(-N // 128)), device="cuda") for _ in range(200)]
    for i in range(200):
        a, sa, w, sw = sets[i % 2]
        moe.grouped_gemm_fp8(handle, a, sa, None, w, sw, outs[i], num_groups=1, N=N, K=K)
        moe.grouped_gate_up_fp8(handle, a, sa, None, w, sw, w, sw, qs[i], ss[i], num_groups=1, H=K, I=N)
    torch.cuda.synchronize()
    for t in (outs, qs, torch.stack(ss)):
        assert not torch.equal(t[0], t[1])
        assert (t[::2] == t[0]).all() and (t[1::2] == t[1]).all()
    for i in range(2):
        a, sa, w, sw = sets[i]
        up = lambda s, n, axis: s.to(F64).repeat_interleave(128, axis).narrow(axis, 0, n)  # noqa: E731
        x = a.view(E4M3).to(F64) * up(sa, K, 1)
        y = (w[0].view(E4M3).to(F64) * up(up(sw[0], N, 0), K, 1)).t()
        # sums of a block's 128 exact products, then of blocks and parts, in fp32 (as test_gpu_fp8 derives it)
        assert ((outs[i].to(F64) - x @ y).abs() <= (128 + nb + 12) * 2.0 ** -23 * (x.abs() @ y.abs()) + 1e-30).all()
