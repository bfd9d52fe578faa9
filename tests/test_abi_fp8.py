"""Argument checks of the balance loss and of the products in E4M3 with scales per block of 128 (no GPU, no launch)."""
import ctypes
import types

import pytest
import torch

import routed_expert_ffn_04_gb300 as moe

P = ctypes.c_void_p
INVALID = moe.MOE_ERR_INVALID_ARG
A = [P(1 << 30 | i << 24) for i in range(12)]  # addresses far apart


@pytest.fixture(scope="module")
def lib():
    return moe.load(build_if_missing=True)


def cfg(**kw):
    return ctypes.byref(moe.make_config(**{**dict(T=64, H=64, E=16, K=2, I=64, I_shared=0, scaling=1.0), **kw}))


def test_balance_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_balance_loss_workspace_size(cfg(), 3, ctypes.byref(n)) == 0 and n.value >= (2 + 3) * 16 * 8
    for seqs in (0, -1, (1 << 20) + 1):
        assert lib.moe_balance_loss_workspace_size(cfg(), seqs, ctypes.byref(n)) == INVALID
    assert lib.moe_balance_loss_workspace_size(cfg(), 1, None) == INVALID
    assert moe.balance_loss_workspace_size(moe.make_config(8192, 64, 192, 8, 64, 0, 1.0)) >= 192 * 8


def test_balance_refusals(lib):
    def loss(score=0, coef=1.0, l=A[0], idx=A[1], seq=A[2], B=2, cnt=A[3], prob=A[4], out=A[5], ws=A[6], size=1 << 20, h=None):
        return lib.moe_balance_loss(h, cfg(), score, coef, l, idx, seq, B, cnt, prob, out, ws, size, None)

    assert loss(size=8) == moe.MOE_ERR_WORKSPACE
    for bad in (dict(score=2), dict(score=-1), dict(coef=float("nan")), dict(coef=float("inf")), dict(l=None), dict(idx=None),
                dict(seq=None), dict(B=0), dict(cnt=None), dict(prob=None), dict(out=None), dict(ws=None), dict(l=P(4100)),
                dict(prob=A[0]), dict(cnt=A[4]), dict(ws=A[1]), dict()):  # dict(): the null handle
        assert loss(**bad) == INVALID

    def grad(score=0, coef=1.0, l=A[0], cnt=A[1], seq=A[2], B=2, d=A[3], add=None, out=A[4]):
        return lib.moe_balance_loss_backward(None, cfg(), score, coef, l, cnt, seq, B, d, add, out, None)

    for bad in (dict(score=2), dict(coef=float("inf")), dict(l=None), dict(cnt=None), dict(seq=None), dict(d=None), dict(out=None),
                dict(out=A[0]), dict(add=P(A[4].value + 16)), dict(B=0), dict(d=P(4100)), dict()):
        assert grad(**bad) == INVALID


def test_balance_token_limit(lib):
    """T up to 2^30 (token indices are 32 bits, and a block's strip of tokens ends past T)."""
    n = ctypes.c_size_t(0)
    for T, ok in ((1 << 30, True), ((1 << 30) + 1, False), ((1 << 31) - 1, False)):
        c = cfg(T=T, K=1, E=1)
        assert (lib.moe_balance_loss_workspace_size(c, 1, ctypes.byref(n)) == 0) is ok
        far = [P(1 << 44), P(1 << 43), *A]
        # Allowed sizes get as far as the workspace's.
        st = lib.moe_balance_loss(None, c, 0, 1.0, far[0], far[1], None, 1, A[0], A[1], A[2], A[3], 8, None)
        assert st == (moe.MOE_ERR_WORKSPACE if ok else INVALID)
        if not ok:
            assert lib.moe_balance_loss_backward(None, c, 0, 1.0, far[0], A[0], None, 1, A[1], None, far[1], None) == INVALID


def test_padded_rows(lib):
    assert moe.fp8_padded_rows(0, 1) == 128 and moe.fp8_padded_rows(127, 3) == 384 and moe.fp8_padded_rows(128, 1) == 256
    for n, G in ((-1, 1), (1, 0), (1, 1025)):
        with pytest.raises(moe.MoEError):
            moe.fp8_padded_rows(n, G)


def test_quantize_refusals(lib):
    q = lambda x=A[0], t=0, b=1, r=8, c=128, sq=0, o=A[1], s=A[2]: lib.moe_quantize_fp8(None, x, t, b, r, c, sq, o, s, None)  # noqa: E731
    for bad in (dict(x=None), dict(o=None), dict(s=None), dict(t=2), dict(b=-1), dict(r=-1), dict(c=0), dict(c=120), dict(o=A[0]),
                dict(s=A[1]), dict(x=P(4100)), dict(b=1 << 40), dict(b=1 << 30, r=1 << 30), dict()):
        assert q(**bad) == INVALID
    c = lambda x=A[0], t=0, G=2, r=8, c=128, off=A[3], o=A[1], s=A[2]: lib.moe_quantize_fp8_columns(None, x, t, G, r, c, off, o, s, None)  # noqa: E731
    for bad in (dict(x=None), dict(o=None), dict(s=None), dict(t=2), dict(G=0), dict(G=1025), dict(r=-1), dict(c=0), dict(c=24),
                dict(off=None), dict(o=A[0]), dict(s=A[3]), dict(c=1 << 17), dict()):
        assert c(**bad) == INVALID


def test_product_refusals(lib):
    def gemm(G=2, r=8, N=128, K=256, tr=0, a=A[0], sa=A[1], off=A[2], w=A[3], sw=A[4], t=0, out=A[5]):
        return lib.moe_grouped_gemm_fp8(None, G, r, N, K, tr, a, sa, off, w, sw, t, out, None)

    for bad in (dict(G=0), dict(G=1025), dict(r=-1), dict(N=0), dict(N=120), dict(K=8), dict(K=1 << 17), dict(a=None), dict(sa=None),
                dict(off=None), dict(w=None), dict(sw=None), dict(out=None), dict(t=5), dict(out=A[0]), dict(out=A[3]), dict(w=P(4100)), dict()):
        assert gemm(**bad) == INVALID

    def gu(G=2, r=8, H=128, I=256, a=A[0], sa=A[1], off=A[2], wg=A[3], sg=A[4], wu=A[5], su=A[6], q=A[7], s=A[8]):
        return lib.moe_grouped_gate_up_fp8(None, G, r, H, I, a, sa, off, wg, sg, wu, su, q, s, None)

    for bad in (dict(G=0), dict(H=24), dict(I=24), dict(a=None), dict(sa=None), dict(off=None), dict(wg=None), dict(sg=None),
                dict(wu=None), dict(su=None), dict(q=None), dict(s=None), dict(q=A[0]), dict(s=A[7]), dict()):
        assert gu(**bad) == INVALID

    def wgrad(G=2, r=8, N=128, K=256, dy=A[0], sd=A[1], a=A[2], sa=A[3], off=A[4], t=0, dw=A[5]):
        return lib.moe_grouped_weight_grad_fp8(None, G, r, N, K, dy, sd, a, sa, off, t, dw, None)

    for bad in (dict(G=0), dict(N=24), dict(K=24), dict(dy=None), dict(sd=None), dict(a=None), dict(sa=None), dict(off=None),
                dict(dw=None), dict(t=3), dict(dw=A[2]), dict()):
        assert wgrad(**bad) == INVALID


H = types.SimpleNamespace(address=None, device=0)


def test_python_refuses_host_tensors():
    c, f, u = moe.make_config(4, 64, 8, 2, 64, 64, 1.0), torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.uint8)
    i = torch.zeros(8, dtype=torch.int32)
    kw = dict(num_groups=1, N=128, K=128)
    for call in (lambda: moe.balance_loss(H, c, f, i, i, f, f, f), lambda: moe.balance_loss(H, c, f, i, i, f, f, f, seq_offsets=i),
                 lambda: moe.balance_loss_backward(H, c, f, i, f, f), lambda: moe.quantize_fp8(H, f, u, f),
                 lambda: moe.quantize_fp8(H, None, u, f), lambda: moe.quantize_fp8_columns(H, f, None, u, f, num_groups=1),
                 lambda: moe.quantize_fp8_columns(H, f, None, u, f, num_groups=0),
                 lambda: moe.grouped_gemm_fp8(H, u, f, None, u, f, f, **kw), lambda: moe.grouped_gemm_fp8(H, u, f, None, u, f, f, num_groups=1, N=128, K=64),
                 lambda: moe.grouped_gemm_fp8(H, u, f, None, u, f, f, num_groups=-1, N=128, K=128),
                 lambda: moe.grouped_gemm_fp8(H, u, f, None, u, f, f, num_groups=1, N=2**40, K=128),
                 lambda: moe.grouped_gate_up_fp8(H, u, f, None, u, f, u, f, u, f, num_groups=1, H=128, I=128),
                 lambda: moe.grouped_weight_grad_fp8(H, u, f, u, f, None, f, rows=4, **kw)):
        with pytest.raises(moe.MoEError) as e:
            call()
        assert e.value.status == INVALID
    with pytest.raises(TypeError):
        moe.balance_loss(H, c, f, i, i, f, f, f, coef="much")


def test_row_limits(lib):
    """Rows up to 2^30: rows and tiles are counted in 32 bits, with every group padded to a multiple of 128. Allowed calls
    get as far as the device, which this handle names wrongly (and they are left out where a device could be found)."""
    wrong = ctypes.create_string_buffer(1 << 16)
    ctypes.memmove(wrong, (1 << 20).to_bytes(4, "little"), 4)
    h = ctypes.cast(wrong, P)
    far = [P((i + 1) << 44) for i in range(9)]
    x, s, off, w, sw, o, s2 = far[:7]
    T = 1 << 30

    def gemm(r, tr=0):
        return lib.moe_grouped_gemm_fp8(h, 2, r, 16, 16, tr, x, s, off, w, sw, 0, o, None)

    def gate_up(r):
        return lib.moe_grouped_gate_up_fp8(h, 2, r, 16, 16, x, s, off, w, sw, far[7], far[8], o, s2, None)

    def wgrad(r):
        return lib.moe_grouped_weight_grad_fp8(h, 2, r, 16, 16, x, s, w, sw, off, 0, o, None)

    def swiglu(r):
        return lib.moe_grouped_swiglu_gemm(h, 2, r, 128, 128, moe.MOE_FP8_BLOCK128, x, s, off, w, far[7], far[8], sw, sw, sw,
                                           o, s2, 1 << 42, None)

    def quantize(r, squares=0, batch=1):
        return lib.moe_quantize_fp8(h, x, 0, batch, r, 16, squares, o, s, None)

    def columns(r):
        return lib.moe_quantize_fp8_columns(h, x, 0, 2, r, 16, off, o, s, None)

    calls = [gemm, lambda r: gemm(r, 1), gate_up, wgrad, swiglu, quantize, lambda r: quantize(r, 1), columns]
    for call in calls:
        for r in (T + 1, 2**31 - 129, 2**31 - 1):
            assert call(r) == INVALID
        if not torch.cuda.is_available():
            assert call(T) == moe.MOE_ERR_CUDA
    assert quantize(1, 1, 1 << 31) == INVALID  # squares
    if not torch.cuda.is_available():
        assert quantize(1, 1, (1 << 31) - 1) == moe.MOE_ERR_CUDA and quantize(1, 0, 1 << 31) == moe.MOE_ERR_CUDA
    for c in (T + 16, 2**31 - 16):
        for sq in (0, 1):
            assert lib.moe_quantize_fp8(h, x, 0, 1, 1, c, sq, o, s, None) == INVALID
    n = ctypes.c_int64(0)
    assert lib.moe_fp8_padded_rows(T, 1024, ctypes.byref(n)) == 0 and n.value == T + 1024 * 128
    assert lib.moe_fp8_padded_rows(T + 1, 1, ctypes.byref(n)) == INVALID
