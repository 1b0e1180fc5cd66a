"""Batches of matrices that do not run side by side: moe_orthogonalize takes them in rounds on one workspace.
Tolerance: one rounding to bf16 (2^-8 of the norm at most) and twice the 1.7e-3 that the iteration's simulated
roundings leave after five steps; steps add theirs (as many fifths of it)."""
import pytest
import torch

import sparse_mixture_experts_16_b200 as moe

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315


def iterate(g, steps=5):
    x = g.double()
    norm = torch.linalg.matrix_norm(x, keepdim=True)
    x = x / torch.where(norm > 0, norm, torch.ones_like(norm))
    for _ in range(steps):
        if x.shape[-2] <= x.shape[-1]:
            G = x @ x.transpose(-1, -2)
            x = A * x + (B * G + C * G @ G) @ x
        else:
            G = x.transpose(-1, -2) @ x
            x = A * x + x @ (B * G + C * G @ G)
    return x


def off(got, ref):
    d, n = torch.linalg.matrix_norm(got.double() - ref), torch.linalg.matrix_norm(ref)
    return float((d / torch.where(n > 0, n, torch.ones_like(n))).max())


def gauss(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("steps", [6, 11, 16])
@pytest.mark.parametrize("shape", [(40, 64, 7168), (5, 65536, 61), (600, 20, 30)], ids=str)
def test_short_sides_with_more_than_five_steps(cuda_device, shape, steps):
    """64 MB of fp32 between the steps' rounds: 36 matrices, 4, and all that there are blocks for"""
    g = gauss(*shape)
    g[shape[0] // 2] = 0
    u, ws = moe.moe_orthogonalize(g, steps=steps)
    assert moe.moe_get_device_error(ws) == 0
    assert (u[shape[0] // 2] == 0).all()
    assert off(u, iterate(g, steps)) < 2.0 ** -8 + 3.4e-3 * steps / 5
