"""moe_orthogonalize on the GPU against the same iteration in 64 bits.

Tolerance, 2-norm: the result is rounded to bf16 once (at most 2^-8 of every value, so at most 2^-8 of the
norm); the fp16 operands of the iteration with X kept to 22 bits are off by at most 1.7e-3 of the norm over
the spectra of a simulation with exactly these roundings (full rank, rank 8 and 64, polynomial and
geometric decay, one huge entry); twice that is allowed: 2^-8 + 3.4e-3.  Singular values between 0 and 1
go through a polynomial whose values lie in [0, 1.2025]."""
import pytest
import torch

import sparse_mixture_experts_16_b200 as moe

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -8 + 3.4e-3
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
    """the largest relative error of a matrix of the batch"""
    d = torch.linalg.matrix_norm(got.double() - ref)
    n = torch.linalg.matrix_norm(ref)
    return float((d / torch.where(n > 0, n, torch.ones_like(n))).max())


def gauss(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


SHAPES = [(1, 1, 1), (2, 1, 50), (2, 50, 1), (3, 8, 8), (3, 7, 5), (2, 31, 33), (2, 65, 64), (3, 129, 200), (2, 257, 96),
          (2, 100, 301), (1, 300, 520), (2, 520, 263), (5, 256, 256), (1, 777, 1301), (1, 1301, 777)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_64_bits(cuda_device, shape, dtype):
    g = gauss(*shape).to(dtype)
    u, ws = moe.moe_orthogonalize(g)
    assert u.dtype == torch.bfloat16 and u.shape == g.shape
    assert moe.moe_get_device_error(ws) == 0
    assert off(u, iterate(g)) < TOL


@pytest.mark.parametrize("kind", ["rank8", "rank64", "decay1", "decay2", "geometric", "spike", "low_rank_and_noise"])
@pytest.mark.parametrize("shape", [(2, 384, 768), (2, 600, 250)], ids=str)
def test_spectra(cuda_device, shape, kind):
    b, m, n = shape
    if kind.startswith("rank"):
        r = int(kind[4:])
        g = gauss(b, m, r) @ gauss(b, r, n, seed=1)
    elif kind == "spike":
        g = gauss(b, m, n)
        g[:, 3, 5] = 1e4
    elif kind == "low_rank_and_noise":
        g = gauss(b, m, 8) @ gauss(b, 8, n, seed=1) + 0.01 * gauss(b, m, n, seed=2)
    else:
        u, s, v = torch.linalg.svd(gauss(b, m, n).double(), full_matrices=False)
        i = torch.arange(s.shape[-1], device="cuda", dtype=torch.float64)
        s = {"decay1": 1 / (i + 1), "decay2": 1 / (i + 1) ** 2, "geometric": 0.97 ** i}[kind]
        g = (u * s @ v).float()
    assert off(moe.moe_orthogonalize(g)[0], iterate(g)) < TOL


@pytest.mark.parametrize("steps", [1, 2, 3, 8, 16])
def test_steps(cuda_device, steps):
    """each step adds its roundings to the last ones: at most steps / 5 of the simulated five"""
    g = gauss(2, 136, 200)
    assert off(moe.moe_orthogonalize(g, steps=steps)[0], iterate(g, steps)) < 2.0 ** -8 + 3.4e-3 * max(1, steps / 5)


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-4, 1e30])
def test_any_magnitude(cuda_device, scale):
    g = gauss(2, 96, 160) * scale
    assert off(moe.moe_orthogonalize(g)[0], iterate(g)) < TOL


def test_zero_nan_and_infinite_matrices_stay_apart(cuda_device):
    g = gauss(6, 70, 90)
    g[1] = 0
    g[3, 2, 5] = float("nan")
    g[4, 60, 80] = float("inf")
    u, _ = moe.moe_orthogonalize(g)
    assert (u[1] == 0).all()
    assert torch.isnan(u[3]).all() and torch.isnan(u[4]).all()
    keep = [0, 2, 5]
    assert off(u[keep], iterate(g[keep])) < TOL


def test_zero_values_in_a_matrix(cuda_device):
    g = gauss(2, 300, 128)
    g[0, 100:] = 0
    g[1, :, 10:] = 0
    u, _ = moe.moe_orthogonalize(g)
    assert off(u, iterate(g)) < TOL
    assert (u[0, 100:] == 0).all() and (u[1, :, 10:] == 0).all()


def test_a_batch_in_several_rounds(cuda_device):
    """more matrices than run side by side; each comes out as it does alone"""
    g = gauss(700, 40, 56)
    u, _ = moe.moe_orthogonalize(g)
    assert off(u, iterate(g)) < TOL
    for i in (0, 591, 592, 699):
        assert off(moe.moe_orthogonalize(g[i])[0][None], iterate(g[i:i + 1])) < TOL


def test_more_dimensions_and_out(cuda_device):
    g = gauss(2, 3, 64, 48)
    out = torch.full((2, 3, 64, 48), 9.0, dtype=torch.bfloat16, device="cuda")
    u, ws = moe.moe_orthogonalize(g, out=out)
    assert u is out and off(out, iterate(g)) < TOL
    assert moe.moe_orthogonalize(g[:0], ws=ws)[0].shape == (0, 3, 64, 48)


def test_same_bits_every_time_and_a_shared_workspace(cuda_device):
    g, h = gauss(2, 200, 600), gauss(1, 600, 130, seed=1)
    need = max(moe.lib().moe_orthogonalize_workspace_size(2, 200, 600),
               moe.lib().moe_orthogonalize_workspace_size(1, 600, 130))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = moe.moe_orthogonalize(g, ws=ws)[0], moe.moe_orthogonalize(h, ws=ws)[0]
    for _ in range(10):
        assert torch.equal(first[0], moe.moe_orthogonalize(g, ws=ws)[0])
        assert torch.equal(first[1], moe.moe_orthogonalize(h, ws=ws)[0])


def test_captured_and_replayed(cuda_device):
    g = gauss(3, 130, 90)
    u, ws = moe.moe_orthogonalize(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out=u, ws=ws)
    for seed in (5, 6):
        g.copy_(gauss(3, 130, 90, seed=seed))
        graph.replay()
        assert off(u, iterate(g)) < TOL


def test_refusals(cuda_device):
    g = gauss(2, 16, 24)
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(g.transpose(1, 2))
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(g.half())
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(g[0, 0])
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(g, out=torch.empty(2, 16, 24, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_orthogonalize(g, steps=0)


def test_an_expert_layer_trained_with_it(cuda_device):
    """permute -> product -> relu -> product -> gradients -> orthogonalised updates, as a training step
    runs them, against the same step in 64 bits on the same 16-bit tensors"""
    T, k, E, D, H = 96, 2, 6, 136, 200
    x = gauss(T, D).bfloat16()
    wg = gauss(E, 192, seed=1).bfloat16()
    idx, p = moe.moe_router_topk(gauss(T, 192, seed=2).bfloat16(), wg, None, k)
    off_ = moe.moe_permute(idx, p, None, E)
    offsets, token = off_["offsets"], off_["perm_token"].long()
    w1, w2 = (gauss(E, H, D, seed=3) * D ** -0.5).bfloat16(), (gauss(E, D, H, seed=4) * H ** -0.5).bfloat16()
    xp = x[token].contiguous()
    h, ws = moe.moe_grouped_gemm(xp, offsets, w1)
    a = h.relu()
    y, _ = moe.moe_grouped_gemm(a, offsets, w2, ws=ws)
    dy = gauss(T * k, D, seed=5).bfloat16()
    da, _ = moe.moe_grouped_gemm_dgrad(dy, offsets, w2, ws=ws)
    dh = torch.where(h > 0, da, torch.zeros_like(da))
    dx, _ = moe.moe_grouped_gemm_dgrad(dh, offsets, w1, ws=ws)
    dw2, ws2 = moe.moe_grouped_gemm_wgrad(dy, a, offsets)
    dw1, _ = moe.moe_grouped_gemm_wgrad(dh, xp, offsets, ws=ws2)
    u1, ws3 = moe.moe_orthogonalize(dw1)
    u2, _ = moe.moe_orthogonalize(dw2, ws=ws3)
    assert all(moe.moe_get_device_error(t) == 0 for t in (ws, ws2, ws3))
    edges = offsets.tolist()
    assert edges[-1] == T * k
    for e in range(E):
        s = slice(edges[e], edges[e + 1])
        rows = edges[e + 1] - edges[e]
        pairs = [(h[s], xp[s], w1[e].T, D), (y[s], a[s], w2[e].T, H), (da[s], dy[s], w2[e], D), (dx[s], dh[s], w1[e], H),
                 (dw2[e], dy[s].T, a[s], rows), (dw1[e], dh[s].T, xp[s], rows)]
        for got, l, r, n in pairs:
            ref, mag = l.double() @ r.double(), l.double().abs() @ r.double().abs()
            # one rounding to the result's type, n + n/16 + 1 truncated additions
            lim = torch.finfo(got.dtype).eps / 2 * ref.abs() + 1.01 * (n + n / 16 + 1) * 2.0 ** -23 * mag
            assert ((got.double() - ref).abs() <= lim + 1e-30).all()
    assert off(u1, iterate(dw1)) < TOL and off(u2, iterate(dw2)) < TOL


SMALL = [(1, 1, 300), (3, 2, 2), (2, 24, 3000), (2, 300, 29), (4, 32, 32), (2, 33, 70), (2, 64, 64), (3, 500, 64),
         (2, 61, 4099), (700, 5, 9), (2, 65, 65)]


@pytest.mark.parametrize("steps", [1, 2, 5, 6, 16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("shape", SMALL, ids=str)
def test_short_sides(cuda_device, shape, dtype, steps):
    """a shorter side of at most 64, and up to five steps, has kernels of its own in fp32: below 1e-3 in their
    simulation, less than the general path's share of the tolerance.  Whatever the steps, the tolerance is
    that of test_steps; a matrix of one row only scales."""
    g = gauss(*shape, seed=7).to(dtype)
    u, ws = moe.moe_orthogonalize(g, steps=steps)
    assert moe.moe_get_device_error(ws) == 0
    assert off(u, iterate(g, steps)) < 2.0 ** -8 + 3.4e-3 * max(1, steps / 5)


@pytest.mark.parametrize("kind", ["rank1", "rank4", "decay1", "decay2", "decay4", "geometric", "spike", "low_rank_and_noise"])
@pytest.mark.parametrize("shape", [(2, 64, 64), (2, 32, 900), (2, 900, 64), (2, 40, 70)], ids=str)
def test_short_sides_of_other_spectra(cuda_device, shape, kind):
    b, m, n = shape
    if kind.startswith("rank"):
        r = int(kind[4:])
        g = gauss(b, m, r) @ gauss(b, r, n, seed=1)
    elif kind == "spike":
        g = gauss(b, m, n)
        g[:, 3, 5] = 1e4
    elif kind == "low_rank_and_noise":
        g = gauss(b, m, 4) @ gauss(b, 4, n, seed=1) + 0.01 * gauss(b, m, n, seed=2)
    else:
        u, s, v = torch.linalg.svd(gauss(b, m, n).double(), full_matrices=False)
        i = torch.arange(s.shape[-1], device="cuda", dtype=torch.float64)
        s = {"decay1": 1 / (i + 1), "decay2": 1 / (i + 1) ** 2, "decay4": 1 / (i + 1) ** 4, "geometric": 0.7 ** i}[kind]
        g = (u * s @ v).float()
    assert off(moe.moe_orthogonalize(g)[0], iterate(g)) < TOL


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e30])
@pytest.mark.parametrize("shape", [(2, 20, 90), (2, 90, 50)], ids=str)
def test_short_sides_of_any_magnitude(cuda_device, shape, scale):
    g = gauss(*shape) * scale
    assert off(moe.moe_orthogonalize(g)[0], iterate(g)) < TOL


def test_short_sides_zero_nan_and_infinite_matrices_stay_apart(cuda_device):
    g = gauss(6, 30, 90)
    g[1] = 0
    g[3, 2, 5] = float("nan")
    g[4, 20, 80] = float("inf")
    u, _ = moe.moe_orthogonalize(g)
    assert (u[1] == 0).all()
    assert torch.isnan(u[3]).all() and torch.isnan(u[4]).all()
    keep = [0, 2, 5]
    assert off(u[keep], iterate(g[keep])) < TOL


def test_short_sides_captured_and_replayed(cuda_device):
    g = gauss(3, 30, 500)
    u, ws = moe.moe_orthogonalize(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out=u, ws=ws)
    for seed in (5, 6):
        g.copy_(gauss(3, 30, 500, seed=seed))
        graph.replay()
        assert off(u, iterate(g)) < TOL
    again, _ = moe.moe_orthogonalize(g, ws=ws)
    assert torch.equal(again, u)
