"""moe_orthogonalize reads what a kernel before it has just written: its own rounds in place, and a weight
gradient whose launch lets the next one start early.  Every call gives the bits that it gives when the GPU was
idle before it."""
import pytest
import torch

import sparse_mixture_experts_16_b200 as moe

pytestmark = pytest.mark.gpu


def gauss(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("steps", [6, 11, 16])
@pytest.mark.parametrize("shape", [(64, 64, 7168), (150, 500, 37)], ids=str)
def test_rounds_in_place_give_the_same_bits(cuda_device, shape, steps):
    """more than five steps of a short side run in rounds, the third of them in place; two batches in turn leave
    other values where the next call's rounds lie"""
    g, h = gauss(*shape), gauss(*shape, seed=1)
    first, ws = moe.moe_orthogonalize(g, steps=steps)
    other, _ = moe.moe_orthogonalize(h, steps=steps, ws=ws)
    first, other = first.clone(), other.clone()
    for _ in range(5):
        assert torch.equal(moe.moe_orthogonalize(g, steps=steps, ws=ws)[0], first)
        assert torch.equal(moe.moe_orthogonalize(h, steps=steps, ws=ws)[0], other)


@pytest.mark.parametrize("N,K", [(48, 1024), (264, 392)])
def test_straight_behind_a_weight_gradient(cuda_device, N, K):
    E, rows = 24, 40
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * rows
    dys = [gauss(E * rows, N, seed=s).bfloat16() for s in range(4)]
    x = gauss(E * rows, K, seed=9).bfloat16()
    dw, ws = moe.moe_grouped_gemm_wgrad(dys[0], x, off)
    u, ws2 = moe.moe_orthogonalize(dw)
    alone = []
    for dy in dys:
        moe.moe_grouped_gemm_wgrad(dy, x, off, out=dw, ws=ws)
        torch.cuda.synchronize()
        moe.moe_orthogonalize(dw, out=u, ws=ws2)
        torch.cuda.synchronize()
        alone.append(u.clone())
    for _ in range(10):
        got = []
        for dy in dys:
            moe.moe_grouped_gemm_wgrad(dy, x, off, out=dw, ws=ws)
            moe.moe_orthogonalize(dw, out=u, ws=ws2)
            got.append(u.clone())
        assert all(torch.equal(a, b) for a, b in zip(got, alone))
