"""Products in E4M3 with one fp32 scale per block of 128: sums shared between thread blocks, over many launches."""
import pytest
import torch

import routed_expert_ffn_04_gb300 as moe

pytestmark = pytest.mark.gpu

E4M3, F32, F64, U8 = torch.float8_e4m3fn, torch.float32, torch.float64, torch.uint8


@pytest.fixture(scope="module")
def handle():
    h = moe.Handle(0)
    yield h
    torch.cuda.synchronize()
    assert h.device_status() == 0
    h.close()


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
