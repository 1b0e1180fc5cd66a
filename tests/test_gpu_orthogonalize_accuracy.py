"""How near moe_orthogonalize comes to the iterate in 64 bits, in the 2-norm, for gradients of experts with few
tokens: low rank, or one direction over a faint rest.  Rounding the 64-bit iterate of such a matrix to bf16
costs little in the 2-norm (its errors point everywhere), so that what the iteration itself adds shows."""
import pytest
import torch

import sparse_mixture_experts_16_b200 as moe

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315


def iterate(g, steps=5):
    x = g.double()
    x = x / torch.linalg.matrix_norm(x, keepdim=True)
    for _ in range(steps):
        if x.shape[-2] <= x.shape[-1]:
            G = x @ x.transpose(-1, -2)
            x = A * x + (B * G + C * G @ G) @ x
        else:
            G = x.transpose(-1, -2) @ x
            x = A * x + x @ (B * G + C * G @ G)
    return x


def off2(got, ref):
    """relative errors of the matrices of a batch in the 2-norm"""
    return torch.linalg.matrix_norm(got.double() - ref, 2) / torch.linalg.matrix_norm(ref, 2)


def gauss(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def over_a_tail(b, m, n, tail):
    u, _, v = torch.linalg.svd(gauss(b, m, n, seed=3).double(), full_matrices=False)
    s = torch.full((u.shape[-1],), tail, dtype=torch.float64, device="cuda")
    s[0] = 1
    return (u * s @ v).float()


# what a simulation of exactly the iteration's roundings leaves before the rounding to bf16, at most, over four
# seeds and five sizes from 65 x 3000 to 384 x 768
SIMULATED = {"rank1": 5.3e-4, "rank4": 6.6e-4, "rank8": 8.2e-4, "low_rank_and_noise": 8.6e-4, "tail": 5.8e-4}


@pytest.mark.parametrize("kind", SIMULATED)
@pytest.mark.parametrize("shape", [(2, 384, 768), (2, 128, 256), (2, 600, 250), (1, 513, 512)], ids=str)
def test_few_directions(cuda_device, shape, kind):
    """A value near its bf16 neighbours' middle may round the other way, never further off: the rounding of
    the 64-bit iterate itself, a tenth more because the 2-norm of random errors varies, and twice the simulation."""
    b, m, n = shape
    if kind == "tail":
        g = over_a_tail(b, m, n, 1e-5)
    else:
        r = int(kind[4:]) if kind.startswith("rank") else 8
        g = gauss(b, m, r) @ gauss(b, r, n, seed=1)
        if kind == "low_rank_and_noise":
            g += 0.01 * gauss(b, m, n, seed=2)
    ref = iterate(g)
    limit = 1.1 * off2(ref.bfloat16(), ref) + 2 * SIMULATED[kind]
    got = off2(moe.moe_orthogonalize(g)[0], ref)
    assert (got <= limit).all(), (got.tolist(), limit.tolist())


@pytest.mark.parametrize("noise", [1e-2, 1e-3])
@pytest.mark.parametrize("shape", [(1, 16, 7168), (300, 16, 7168), (300, 7168, 60), (512, 8, 65536)], ids=str)
def test_short_sides_whatever_the_batch(cuda_device, shape, noise):
    """One direction and noise, a short side of at most 64: a simulation of the kernels' fp32 steps, its Gram
    sums drained into 64 bits every 64 terms, leaves 5.4e-4 of the Frobenius norm at most, whatever the
    length.  One fp32 chain over the long side would leave 4e-3 to 1.2e-2.  Rounding to bf16: that of the
    64-bit iterate, with a hundredth for roundings that go the other way."""
    b, m, n = shape
    g = (gauss(b, m, 1) @ gauss(b, 1, n, seed=1)).add_(gauss(b, m, n, seed=2), alpha=noise).bfloat16()
    u, ws = moe.moe_orthogonalize(g)
    assert moe.moe_get_device_error(ws) == 0
    for i in {0, b // 2, b - 1}:
        ref = iterate(g[i])
        size = torch.linalg.matrix_norm(ref)
        rounding = torch.linalg.matrix_norm(ref.bfloat16().double() - ref) / size
        got = torch.linalg.matrix_norm(u[i].double() - ref) / size
        assert got <= 1.01 * rounding + 2 * 5.4e-4, (i, float(got), float(rounding))
