"""Products in E4M3 with one fp32 scale per block of 128, their quantisers and the weights' gradient, against plain
definitions in 64 bits.

Tolerances. A result is sum_kb s_kb P_kb with P_kb a sum of 128 exact products in fp32 (each addition off by at most
2^-23 of the running sum of magnitudes, rounding or truncating), times a factor rounded twice and added in fp32:
|error| <= (128 + blocks + 4) 2^-23 S, S the same sum of magnitudes; then one rounding of the output, 2^-8 relative for
bf16. A code is off by half a step: 2^-4 relative, or 2^-10 of the scale near 0."""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe

pytestmark = pytest.mark.gpu

BLOCK = 128
U8, F32, BF16, F64 = torch.uint8, torch.float32, torch.bfloat16, torch.float64
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def handle():
    h = moe.Handle(0)
    yield h
    torch.cuda.synchronize()
    assert h.device_status() == 0
    h.close()


def nblocks(n):
    return -(-n // BLOCK)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(g, *shape):
    return (130.0 * torch.randn(shape, device="cuda", generator=g)).clamp(-448, 448).to(E4M3).view(U8)


def scales(g, *shape, std=0.01):
    return std * (0.5 + torch.rand(shape, device="cuda", generator=g))


def val(q):
    return q.view(E4M3).to(F64)


def spread(s, n, axis):
    return s.to(F64).repeat_interleave(BLOCK, axis).narrow(axis, 0, n)


def rows64(q, s):
    return val(q) * spread(s, q.shape[1], 1)


def squares64(q, s):
    return val(q) * spread(spread(s, q.shape[-2], -2), q.shape[-1], -1)


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def bound(S, kb):
    return (BLOCK + kb + 4) * 2.0 ** -23 * S


def close(got, ref, S, kb, what):
    u = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    err = (got.to(F64) - ref).abs()
    tol = bound(S, kb) * (1 + u) + u * ref.abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err - tol).max()):.3e} of {float(ref.abs().max()):.3e}"


# ---------------------------------------------------------------- quantisers
def quantize64(x, height, width):
    """Scales in fp32 as defined, codes of the quotients rounded to fp32 (as a division gives)."""
    R, C = x.shape
    full = torch.zeros(-(-R // height) * height, -(-C // width) * width, dtype=F32, device="cuda")
    full[:R, :C] = x.to(F32)
    b = full.reshape(full.shape[0] // height, height, full.shape[1] // width, width)
    amax = b.abs().amax((1, 3))
    s = (amax / torch.full_like(amax, 448.0)).clamp(min=2.0 ** -126)  # by a tensor: by a number, torch multiplies by 1 / 448
    q = (b / s[:, None, :, None]).clamp(-448, 448).to(E4M3).view(U8).reshape(full.shape)
    return q[:R, :C], s


def inputs(g, kind, R, C, dtype):
    x = torch.randn((R, C), device="cuda", generator=g)
    if kind == "wide":
        x *= torch.exp2(torch.randint(-60, 60, (R, C), device="cuda", generator=g).float())
    elif kind == "tiny":
        x *= 2.0 ** -133
    elif kind == "zeros":
        x *= (torch.rand((R, C), device="cuda", generator=g) < 0.005)
    return x.to(dtype)


@pytest.mark.parametrize("kind", ["normal", "wide", "tiny", "zeros"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R, C", [(1, 16), (1, 128), (7, 144), (129, 400), (300, 1024), (64, 4096)])
@pytest.mark.parametrize("squares", [False, True])
def test_quantize(handle, squares, R, C, dtype, kind):
    x = inputs(gen(R + C), kind, R, C, dtype)
    q = torch.full((R, C), 0xA5, dtype=U8, device="cuda")
    s = torch.full((nblocks(R) if squares else R, nblocks(C)), -1.0, device="cuda")
    moe.quantize_fp8(handle, x, q, s, squares=squares)
    qr, sr = quantize64(x, BLOCK if squares else 1, BLOCK)
    assert torch.equal(s, sr)
    # -0 and 0 stand for the same; every code is that of the fp32 quotient
    assert torch.equal(q.view(E4M3).float(), qr.view(E4M3).float())


def test_quantize_batch(handle):
    x = torch.randn((3, 200, 272), device="cuda", generator=gen(5)).to(BF16)
    q, s = torch.empty(x.shape, dtype=U8, device="cuda"), torch.empty((3, 2, 3), device="cuda")
    moe.quantize_fp8(handle, x, q, s, squares=True)
    for i in range(3):
        qr, sr = quantize64(x[i], BLOCK, BLOCK)
        assert torch.equal(s[i], sr) and torch.equal(q[i], qr)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_not_finite(handle, dtype, bad):
    """The block stands for NaN throughout, the others for what they were."""
    x = torch.randn((256, 256), device="cuda", generator=gen(6)).to(dtype)
    x[3, 130] = bad
    clean = x.clone()
    clean[3, 130] = 0
    off = offsets_of([256])
    for form, height, width, where in (("rows", 1, 128, (slice(3, 4), slice(128, 256))),
                                       ("squares", 128, 128, (slice(0, 128), slice(128, 256))),
                                       ("columns", 128, 1, (slice(0, 128), slice(130, 131)))):
        rows = moe.fp8_padded_rows(256, 1) if form == "columns" else 256
        q = torch.zeros((rows, 256), dtype=U8, device="cuda")
        s = torch.zeros((-(-rows // height), -(-256 // width)), device="cuda")
        if form == "columns":
            moe.quantize_fp8_columns(handle, x, off, q, s, num_groups=1)
        else:
            moe.quantize_fp8(handle, x, q, s, squares=form == "squares")
        v = val(q[:256]) * s[: 256 // height].to(F64).repeat_interleave(height, 0).repeat_interleave(width, 1)
        nan = torch.zeros((256, 256), dtype=torch.bool, device="cuda")
        nan[where] = True
        assert torch.equal(v.isnan(), nan)
        qr, _ = quantize64(clean, height, width)
        assert torch.equal(q[:256][~nan], qr[~nan])


COUNTS = [[1], [0, 0, 5], [128, 0, 129, 1, 127], [300, 17, 0, 256], [1] * 40, [0, 777, 0]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C", [16, 400, 1024])
def test_quantize_columns(handle, C, dtype, counts):
    """Groups padded to 128 rows; rows behind the last group are not read and blocks behind it not written."""
    rows, G = sum(counts) + 3, len(counts)
    x = inputs(gen(rows + C), "wide", rows, C, dtype)
    x[sum(counts):] = float("nan")
    P = moe.fp8_padded_rows(rows, G)
    assert P == (rows // 128 + G) * 128
    q = torch.full((P, C), 0xA5, dtype=U8, device="cuda")
    s = torch.full((P // 128, C), -1.0, device="cuda")
    moe.quantize_fp8_columns(handle, x, offsets_of(counts), q, s, num_groups=G)
    at = r = 0
    for n in counts:
        if n:
            qr, sr = quantize64(x[r:r + n], BLOCK, 1)
            assert torch.equal(s[at // 128:at // 128 + nblocks(n)], sr)
            assert torch.equal(q[at:at + n].view(E4M3).float(), qr.view(E4M3).float())
            assert (q[at + n:at + nblocks(n) * 128] == 0).all()
        r += n
        at += nblocks(n) * 128
    assert (q[at:] == 0xA5).all() and (s[at // 128:] == -1.0).all()


# ---------------------------------------------------------------- products
def product(handle, counts, N, K, transposed, out_dtype, seed=0, dense=False):
    g, G, used = gen(seed), len(counts), sum(counts)
    rows = used + (0 if dense else 2)
    a, sa = codes(g, rows, K), scales(g, rows, nblocks(K))
    A, B = (K, N) if transposed else (N, K)
    w, sw = codes(g, G, A, B), scales(g, G, nblocks(A), nblocks(B))
    a[used:] = 0x7F  # rows of no group may hold anything
    off = None if dense else offsets_of(counts)
    out = torch.full((rows, N), 7.0, dtype=out_dtype, device="cuda")
    moe.grouped_gemm_fp8(handle, a, sa, off, w, sw, out, num_groups=G, N=N, K=K, transposed=transposed)
    assert (out[used:] == 7.0).all()
    r = 0
    for i, n in enumerate(counts):
        x, y = rows64(a[r:r + n], sa[r:r + n]), squares64(w[i], sw[i])
        y = y if transposed else y.t()
        close(out[r:r + n], x @ y, x.abs() @ y.abs(), nblocks(K), f"group {i} of {n}")
        r += n
    return out


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("counts, N, K", [
    ([1], 128, 128), ([1], 16, 16), ([3, 0, 2], 48, 80), ([17, 40, 0, 70, 129], 256, 384), ([256, 257, 0, 512, 31], 272, 144),
    ([100], 1536, 4096), ([5] * 30, 400, 656), ([0, 0], 128, 128), ([33], 128, 4240)])
def test_product(handle, counts, N, K, out_dtype, transposed):
    product(handle, counts, N, K, transposed, out_dtype)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", [1, 7, 64, 130, 1000])
def test_dense_product(handle, rows, transposed):
    """offsets None: one group of all rows."""
    product(handle, [rows], 512, 1024, transposed, BF16, dense=True)


FEW = [([1], 512, 4096), ([33], 272, 1616), ([128], 256, 2048), ([129], 1536, 4096), ([0, 0, 3, 0, 70, 0, 0], 256, 1920),
       ([296], 400, 3728), ([130, 0, 200], 512, 3600), ([3, 9], 272, 528), ([250, 6, 128], 2064, 2048),
       ([20], 272, 1616), ([50], 272, 3728), ([5, 0, 40], 2304, 2704), ([1] * 10, 256, 1360), ([62], 512, 3088)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("counts, N, K", FEW)
def test_few_tiles(handle, counts, N, K, out_dtype, transposed):
    """Few tiles and a long reduction: parts of it on several SMs, of like and unlike lengths."""
    product(handle, counts, N, K, transposed, out_dtype)


def test_few_tiles_same_bits(handle):
    """Sums exchanged between thread blocks: launches back to back, in a graph and on two streams give the same bits."""
    g, rows, N, K = gen(21), 40, 512, 4096
    a, sa, w, sw = codes(g, rows, K), scales(g, rows, 32), codes(g, 1, N, K), scales(g, 1, 4, 32)
    wu, su = codes(g, 1, N, K), scales(g, 1, 4, 32, std=2e-4)
    first = torch.empty((rows, N), dtype=F32, device="cuda")
    fq, fs = torch.empty((rows, N), dtype=U8, device="cuda"), torch.empty((rows, 4), device="cuda")
    outs, qs, ss = torch.zeros((30, rows, N), device="cuda"), torch.zeros((30, rows, N), dtype=U8, device="cuda"), torch.zeros((30, rows, 4), device="cuda")
    h2 = moe.Handle(0)

    def call(h, o, q, s):
        moe.grouped_gemm_fp8(h, a, sa, None, w, sw, o, num_groups=1, N=N, K=K)
        moe.grouped_gate_up_fp8(h, a, sa, None, wu, su, wu, su, q, s, num_groups=1, H=K, I=N)

    call(handle, first, fq, fs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(10):
            call(handle, outs[i], qs[i], ss[i])
    graph.replay()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(10, 30):
        with torch.cuda.stream(streams[i % 2]):
            call(handle if i % 2 else h2, outs[i], qs[i], ss[i])
    torch.cuda.synchronize()
    for i in range(30):
        assert torch.equal(outs[i], first) and torch.equal(qs[i], fq) and torch.equal(ss[i], fs)
    assert handle.device_status() == 0 and h2.device_status() == 0


def test_many_groups(handle):
    product(handle, [(i * 7) % 5 for i in range(1024)], 128, 256, False, BF16)


def test_many_tiles_per_pair(handle):
    """More tiles than SMs, several rounds of every ring."""
    product(handle, [400, 0, 300, 513], 4096, 1536, False, F32)
    product(handle, [400, 0, 300, 513], 4096, 1536, True, BF16)


def test_no_rows(handle):
    w, sw = torch.zeros((2, 128, 128), dtype=U8, device="cuda"), torch.ones((2, 1, 1), device="cuda")
    e = lambda dt, c: torch.empty((0, c), dtype=dt, device="cuda")  # noqa: E731
    moe.grouped_gemm_fp8(handle, e(U8, 128), e(F32, 1), offsets_of([0, 0]), w, sw, e(BF16, 128), num_groups=2, N=128, K=128)
    moe.grouped_gate_up_fp8(handle, e(U8, 128), e(F32, 1), offsets_of([0, 0]), w, sw, w, sw, e(U8, 128), e(F32, 1),
                            num_groups=2, H=128, I=128)


def test_nan_stays_in_its_row_and_group(handle):
    """A NaN code of a row reaches that row alone; one of an expert's weights reaches that expert's rows alone, also
    where a block of 128 reaches past the matrix (N, K not multiples of 128)."""
    g, counts, N, K = gen(3), [40, 50, 60], 144, 176
    a, sa, w, sw = codes(g, 150, K), scales(g, 150, 2), codes(g, 3, N, K), scales(g, 3, 2, 2)
    for transposed in (False, True):
        A, B = (K, N) if transposed else (N, K)
        w2 = w.reshape(3, A, B).clone()
        a2 = a.clone()
        a2[10, 5] = 0x7F
        w2[2] = 0x7F
        out = torch.empty((150, N), dtype=F32, device="cuda")
        moe.grouped_gemm_fp8(handle, a2, sa, offsets_of(counts), w2, sw, out, num_groups=3, N=N, K=K, transposed=transposed)
        want = torch.zeros(150, dtype=torch.bool, device="cuda")
        want[10] = True
        want[90:] = True
        assert torch.equal(out.isnan().any(1), want) and out[want].isnan().all()


# ---------------------------------------------------------------- gate and up
@pytest.mark.parametrize("counts, H, I", [([1], 128, 128), ([1], 16, 48), ([3, 0, 70, 129], 256, 384), ([300, 31, 256], 400, 272),
                                          ([64], 4096, 1536), ([5] * 30, 128, 144)])
def test_gate_up(handle, counts, H, I):
    g, G, used = gen(H + I), len(counts), sum(counts)
    rows = used + 2
    a, sa = codes(g, rows, H), scales(g, rows, nblocks(H))
    wg, wu = codes(g, G, I, H), codes(g, G, I, H)
    sg, su = scales(g, G, nblocks(I), nblocks(H), std=2e-4), scales(g, G, nblocks(I), nblocks(H), std=2e-4)
    a[used:] = 0x7F
    q = torch.full((rows, I), 0xA5, dtype=U8, device="cuda")
    s = torch.full((rows, nblocks(I)), -1.0, device="cuda")
    moe.grouped_gate_up_fp8(handle, a, sa, offsets_of(counts), wg, sg, wu, su, q, s, num_groups=G, H=H, I=I)
    assert (q[used:] == 0xA5).all() and (s[used:] == -1.0).all()
    r, kb = 0, nblocks(H)
    for i, n in enumerate(counts):
        x = rows64(a[r:r + n], sa[r:r + n])
        yg, yu = squares64(wg[i], sg[i]).t(), squares64(wu[i], su[i]).t()
        gate, up = x @ yg, x @ yu
        dg, du = bound(x.abs() @ yg.abs(), kb), bound(x.abs() @ yu.abs(), kb)
        act = gate * torch.sigmoid(gate)
        h = act * up
        # |silu'| <= 1.1; exp, the quotient and two products in fp32
        dh = 1.1 * dg * up.abs() + du * act.abs() + 1.1 * dg * du + 2.0 ** -20 * (1 + gate.abs() / 8) * h.abs()
        sc = s[r:r + n].to(F64)
        pad = nblocks(I) * BLOCK - I
        amax = torch.nn.functional.pad(h.abs(), (0, pad)).reshape(n, nblocks(I), BLOCK).amax(2)
        damax = torch.nn.functional.pad(dh, (0, pad)).reshape(n, nblocks(I), BLOCK).amax(2)
        assert ((sc - amax / 448).abs() <= damax / 448 + 2.0 ** -22 * sc).all()
        back = val(q[r:r + n]) * spread(s[r:r + n], I, 1)
        tol = dh * (1 + 2.0 ** -4) + 2.0 ** -4 * h.abs() + spread(s[r:r + n], I, 1) * 2.0 ** -10
        assert ((back - h).abs() <= tol).all(), f"group {i}: {float(((back - h).abs() - tol).max())}"
        r += n


@pytest.mark.parametrize("counts, I, H", FEW)
def test_gate_up_few_tiles(handle, counts, I, H):
    test_gate_up(handle, counts, H, I)


def test_gate_up_small_and_large_groups_in_turn(handle):
    """Tiles of up to 128 rows and higher ones by turns in the same thread blocks, several of each."""
    test_gate_up(handle, [20, 200, 128, 129] * 20, 128, 512)


# ---------------------------------------------------------------- weights' gradient
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("counts, N, K", [([1], 16, 16), ([0, 5, 0], 48, 80), ([128, 1, 300, 0, 129], 272, 400), ([1000], 256, 512),
                                          ([4] * 50, 144, 128), ([0], 128, 128), ([700, 900], 1536, 1024)])
def test_weight_grad(handle, counts, N, K, out_dtype):
    g, G, rows = gen(N + K), len(counts), sum(counts)
    dy = torch.randn((rows, N), device="cuda", generator=g).to(BF16)
    a = torch.randn((rows, K), device="cuda", generator=g).to(BF16)
    off, P = offsets_of(counts), moe.fp8_padded_rows(rows, G)
    qs = []
    for x, C in ((dy, N), (a, K)):
        # blocks behind the last group hold anything
        q, s = torch.full((P, C), 0x7F, dtype=U8, device="cuda"), torch.full((P // 128, C), float("nan"), device="cuda")
        if rows:
            moe.quantize_fp8_columns(handle, x, off, q, s, num_groups=G)
        qs += [q, s]
    dw = torch.full((G, N, K), 7.0, dtype=out_dtype, device="cuda")
    moe.grouped_weight_grad_fp8(handle, *qs, off, dw, rows=rows, num_groups=G, N=N, K=K)
    at = 0
    for i, n in enumerate(counts):
        m = nblocks(n) * 128
        x, y = (val(q[at:at + m]) * spread(s[at // 128:(at + m) // 128], m, 0) for q, s in (qs[:2], qs[2:]))
        close(dw[i], x.t() @ y, x.abs().t() @ y.abs(), max(1, nblocks(n)), f"group {i} of {n}")
        at += m


def test_offsets_that_fall_stay_inside(handle):
    """Not allowed, and not refused as the offsets are on the device: the groups ask for more blocks than there are. What
    is read and written stays inside the tensors."""
    off, rows, N, K = torch.tensor([0, 300, 0, 300, 0, 300], dtype=torch.int32, device="cuda"), 300, 128, 256
    P = moe.fp8_padded_rows(rows, 5)
    assert P // 128 < 3 * nblocks(rows)
    qs = []
    for C in (N, K):
        q, s = torch.full((P + 1, C), 0xA5, dtype=U8, device="cuda"), torch.full((P // 128 + 1, C), -1.0, device="cuda")
        moe.quantize_fp8_columns(handle, torch.ones((rows, C), dtype=BF16, device="cuda"), off, q[:P], s[:P // 128], num_groups=5)
        assert (q[P:] == 0xA5).all() and (s[P // 128:] == -1.0).all()
        qs += [q[:P], s[:P // 128]]
    dw = torch.full((6, N, K), 7.0, device="cuda")
    moe.grouped_weight_grad_fp8(handle, *qs, off, dw[:5], rows=rows, num_groups=5, N=N, K=K)
    torch.cuda.synchronize()
    assert (dw[5] == 7.0).all() and (dw[1] == 0).all() and (dw[3] == 0).all()


def test_gradient_against_differences(handle):
    """L = <out, v> of out = a w^T: the products' gradients against central differences of the 64-bit forward of the
    values that the codes stand for."""
    g, n, N, K = gen(9), 96, 128, 256
    x, wt, v = (torch.randn(s, device="cuda", generator=g) for s in ((n, K), (N, K), (n, N)))
    a, sa = torch.empty((n, K), dtype=U8, device="cuda"), torch.empty((n, 2), device="cuda")
    w, sw = torch.empty((1, N, K), dtype=U8, device="cuda"), torch.empty((1, 1, 2), device="cuda")
    dy, sdy = torch.empty((n, N), dtype=U8, device="cuda"), torch.empty((n, 1), device="cuda")
    moe.quantize_fp8(handle, x, a, sa)
    moe.quantize_fp8(handle, wt, w, sw, squares=True)
    moe.quantize_fp8(handle, v, dy, sdy)
    da = torch.empty((n, K), device="cuda")
    moe.grouped_gemm_fp8(handle, dy, sdy, None, w, sw, da, num_groups=1, N=K, K=N, transposed=True)
    P = moe.fp8_padded_rows(n, 1)
    cols = [t for X, C in ((v, N), (x, K)) for t in (torch.zeros((P, C), dtype=U8, device="cuda"), torch.zeros((P // 128, C), device="cuda"))]
    off = offsets_of([n])
    moe.quantize_fp8_columns(handle, v, off, cols[0], cols[1], num_groups=1)
    moe.quantize_fp8_columns(handle, x, off, cols[2], cols[3], num_groups=1)
    dw = torch.empty((1, N, K), device="cuda")
    moe.grouped_weight_grad_fp8(handle, *cols, off, dw, rows=n, num_groups=1, N=N, K=K)
    va, vw, vv = rows64(a, sa), squares64(w[0], sw[0]), rows64(dy, sdy)
    ca, cv = (val(q[:n]) * s[:1].to(F64) for q, s in ((cols[2], cols[3]), (cols[0], cols[1])))
    f = lambda A, W, V: ((A @ W.t()) * V).sum()  # noqa: E731
    for i, j in ((0, 0), (17, 100), (95, 255)):
        e = torch.zeros_like(va)
        e[i, j] = 0.5
        d = f(va + e, vw, vv) - f(va - e, vw, vv)  # linear: exact
        assert abs(float(da[i, j]) - float(d)) <= float(bound(vv[i].abs() @ vw[:, j].abs(), 1)) + 1e-9
    for i, j in ((0, 0), (64, 3), (127, 255)):
        e = torch.zeros_like(vw)
        e[i, j] = 0.5
        d = f(ca, vw + e, cv) - f(ca, vw - e, cv)
        assert abs(float(dw[0, i, j]) - float(d)) <= float(bound(cv[:, i].abs() @ ca[:, j].abs(), 1)) + 1e-9


# ---------------------------------------------------------------- streams, graphs, refusals
def test_same_bits_and_streams(handle):
    """The same call gives the same bits, on another stream, in a replayed graph, and beside itself on two streams."""
    args = dict(counts=[300, 0, 77, 256], N=512, K=768, transposed=False, out_dtype=BF16)
    first = product(handle, **args)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert torch.equal(product(handle, **args), first)
    g, used = gen(0), 633
    a, sa, w, sw = codes(g, used + 2, 768), scales(g, used + 2, 6), codes(g, 4, 512, 768), scales(g, 4, 4, 6)
    off = offsets_of(args["counts"])
    outs = [torch.zeros((used + 2, 512), dtype=BF16, device="cuda") for _ in range(3)]
    h2 = moe.Handle(0)
    call = lambda h, o, st=None: moe.grouped_gemm_fp8(h, a, sa, off, w, sw, o, num_groups=4, N=512, K=768, stream=st)  # noqa: E731
    torch.cuda.synchronize()
    s2 = torch.cuda.Stream()
    for _ in range(5):
        call(handle, outs[0], s)
        call(h2, outs[1], s2)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(handle, outs[2])
        call(handle, outs[2])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][:used], outs[1][:used]) and torch.equal(outs[0][:used], outs[2][:used])
    assert h2.device_status() == 0


def test_refused_tensors(handle):
    g = gen(1)
    a, sa, w, sw = codes(g, 8, 256), scales(g, 8, 2), codes(g, 1, 128, 256), scales(g, 1, 1, 2)
    out = torch.empty((8, 128), dtype=BF16, device="cuda")
    kw = dict(num_groups=1, N=128, K=256)
    ok = lambda **k: moe.grouped_gemm_fp8(handle, k.get("a", a), k.get("sa", sa), None, k.get("w", w), k.get("sw", sw),  # noqa: E731
                                          k.get("out", out), **{**kw, **k.get("kw", {})})
    ok()
    for k in (dict(a=a.float()), dict(a=a[:, ::2]), dict(sa=sa[:, :1]), dict(sa=sa.to(BF16)), dict(w=w[:, :64]), dict(sw=sw.cpu()),
              dict(out=out.half()), dict(out=out[:4]), dict(kw=dict(K=248)), dict(kw=dict(num_groups=2)), dict(kw=dict(N=120)),
              dict(out=a.view(BF16))):
        with pytest.raises(moe.MoEError) as e:
            ok(**k)
        assert e.value.status == moe.MOE_ERR_INVALID_ARG
