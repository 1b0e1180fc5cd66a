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


TOL = 2.0 ** -8 + 3.4e-3


@pytest.mark.parametrize("shape", [(1303, 65, 73), (700, 80, 65), (30, 96, 65536), (24, 65536, 90)], ids=str)
def test_other_sides_in_several_rounds(cuda_device, shape):
    """592 matrices at a time, dealt evenly (435, 435 and 433, where the second round's results start on an odd
    element; 350 twice), or as many as 768 MB hold"""
    b = shape[0]
    g = gauss(*shape)
    g[b // 2] = 0
    u, ws = moe.moe_orthogonalize(g)
    assert moe.moe_get_device_error(ws) == 0
    assert (u[b // 2] == 0).all()
    some = range(b) if b > 100 else (0, b // 2 - 1, b // 2 + 1, b - 1)
    ref = iterate(g[list(some)])
    assert off(u[list(some)], ref) < TOL
    for i in (0, b - 1):
        alone = g[i:i + 1].clone()  # on 16 bytes
        assert off(moe.moe_orthogonalize(alone)[0], iterate(alone)) < TOL


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 65, 65536), (2, 65536, 66), (1, 130, 65521), (1, 65535, 257), (1, 4100, 4211)], ids=str)
def test_long_sides(cuda_device, shape, dtype):
    g = gauss(*shape).to(dtype)
    u, ws = moe.moe_orthogonalize(g)
    assert moe.moe_get_device_error(ws) == 0
    assert off(u, iterate(g)) < TOL


@pytest.mark.parametrize("shape", [(3, 70, 90), (3, 90, 70), (2, 129, 257), (2, 300, 136)], ids=str)
def test_rows_behind_the_last_matrix_are_left_as_they_were(cuda_device, shape):
    """the last step stores rows of any length, two bytes or sixteen at a time"""
    b, m, n = shape
    big = torch.full((b * m * n + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    g = gauss(*shape)
    out = big[:b * m * n].view(shape)
    moe.moe_orthogonalize(g, out=out)
    assert (big[b * m * n:] == 7.0).all() and off(out, iterate(g)) < TOL


def test_results_past_32_bits(cuda_device):
    """2^31 elements and more: 515 matrices of [2048, 2048] in bf16, more than 4 GiB; the last and those around
    2^31 elements are looked at"""
    b, m, n = 515, 2048, 2048
    g = torch.empty(b, m, n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(4))
    u, ws = moe.moe_orthogonalize(g)
    assert moe.moe_get_device_error(ws) == 0
    for i in (0, 511, 512, 514):
        assert off(u[i:i + 1], iterate(g[i:i + 1])) < TOL
