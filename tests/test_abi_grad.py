"""Host-side argument checks of the entry points around the layer and of its gradient (no GPU, no launch)."""
import ctypes

import pytest

import routed_expert_ffn_04_gb300 as moe

P = ctypes.c_void_p
INV, WS, UNSUP = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_WORKSPACE, moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return moe.load(build_if_missing=True)


def _cfg(**kw):
    d = dict(T=64, H=4096, E=192, K=8, I=1536, I_shared=1536, scaling=2.826)
    d.update(kw)
    return moe.make_config(**d)


def test_add_rmsnorm_checks(lib):
    def call(rows=4, H=64, rt=0, x=256, res=512, w=768, eps=1e-5, ho=1024, out=1280, q=None, s=None, rstd=None):
        p = lambda v: None if v is None else P(v)  # noqa: E731
        return lib.moe_add_rmsnorm(None, rows, H, rt, p(x), p(res), p(w), eps, p(ho), p(out), p(q), p(s), p(rstd), None)

    for kw in (dict(rows=-1), dict(H=0), dict(H=16385), dict(rt=2), dict(x=None), dict(w=None), dict(out=None),
               dict(q=2048), dict(s=2048), dict(q=2048, s=4096, H=40), dict(eps=float("nan")), dict(eps=-1.0),
               dict(eps=float("inf")), dict(x=264), dict(rstd=2052), dict(rows=1 << 31)):
        assert call(**kw) == INV, kw
    assert call() == INV  # all is well but the null handle


def test_add_rmsnorm_backward_checks(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_add_rmsnorm_backward_workspace_size(100, 4096, ctypes.byref(n)) == moe.MOE_OK
    assert n.value >= 100 * 4096 * 4
    assert moe.add_rmsnorm_backward_workspace_size(1 << 20, 4096) < 8 << 20  # does not grow with the rows
    for rows, H in ((-1, 64), (4, 0), (4, 16385)):
        assert lib.moe_add_rmsnorm_backward_workspace_size(rows, H, ctypes.byref(n)) == INV
    need = moe.add_rmsnorm_backward_workspace_size(100, 64)

    def call(dout=256, h=512, w=768, rstd=1024, dh=1280, dw=1536, ws=4096, wsb=need):
        p = lambda v: None if v is None else P(v)  # noqa: E731
        return lib.moe_add_rmsnorm_backward(None, 100, 64, 0, p(dout), None, p(h), p(w), p(rstd), p(dh), None, p(dw),
                                            p(ws), wsb, None)

    for kw in (dict(dout=None), dict(h=None), dict(rstd=None), dict(dh=None), dict(ws=None), dict(dh=1284)):
        assert call(**kw) == INV, kw
    assert call(wsb=need - 1) == WS
    assert call(dw=None, ws=None, wsb=0) == INV  # no workspace needed: the null handle is what is left


def test_dispatch_gradient_checks(lib):
    c = _cfg()
    a = [P(256 * (i + 1)) for i in range(9)]  # dout, y, w, f2p, idx, logits, dy, dw, dlogits
    call = lambda a, c=c: lib.moe_combine_backward(None, ctypes.byref(c), *a, None)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8):  # a missing one (4, 5 and 8 come together)
        assert call(a[:i] + [None] + a[i + 1:]) == INV, i
    assert call(a[:5] + [a[8]] + a[6:]) == INV  # dlogits over logits
    assert call([P(260)] + a[1:]) == INV
    assert call(a, _cfg(K=0)) == INV
    assert lib.moe_route_backward(None, ctypes.byref(c), a[0], a[1], a[2], a[2], None) == INV
    assert lib.moe_permute_backward(None, ctypes.byref(c), a[0], a[1], None, a[0], None) == INV
    assert lib.moe_permute_backward(None, None, a[0], a[1], None, a[2], None) == INV


def test_grouped_backward_checks(lib):
    n = ctypes.c_size_t(0)
    size = lambda *a: lib.moe_grouped_gemm_backward_workspace_size(*a, ctypes.byref(n))  # noqa: E731
    assert size(100, 4, 256, 128, 0) == moe.MOE_OK and n.value >= 100 * 128 * 10
    assert size(100, 4, 256, 128, 1) == UNSUP and size(100, 4, 256, 128, 7) == INV
    for bad in ((-1, 4, 256, 128, 0), (1, 0, 256, 128, 0), (1, 1025, 256, 128, 0), (1, 1, 96, 128, 0), (1, 1, 128, 32, 0)):
        assert size(*bad) == INV
    size(100, 4, 256, 128, 0)

    def call(g=4, rows=100, H=256, I=128, dt=0, a=256, dy=512, off=768, w=1024, da=2048, dw=(4096, 8192, 16384),
             ws=65536, wsb=n.value):
        p = lambda v: None if v is None else P(v)  # noqa: E731
        return lib.moe_grouped_swiglu_backward(None, g, rows, H, I, dt, p(a), p(dy), p(off), p(w), p(w), p(w), p(da),
                                               *[p(x) for x in dw], p(ws), wsb, None)

    for kw in (dict(a=None), dict(dy=None), dict(off=None), dict(w=None), dict(ws=None), dict(dw=(None, 256, 512)),
               dict(da=None, dw=(None, None, None)), dict(H=100), dict(a=264), dict(g=0), dict(dt=5)):
        assert call(**kw) == INV, kw
    assert call(wsb=100) == WS and call(dt=2) == UNSUP
    assert call() == INV  # the null handle
