"""Calls with ``stream``: what they are given may be let go of while the stream has not come to them yet."""
import pytest
import torch

import sparse_mixture_experts_16_b200 as moe

pytestmark = pytest.mark.gpu


def gauss(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


CALLS = ["gemm", "dgrad", "wgrad", "orthogonalize"]


def run(name, tensors, **kw):
    f = {"gemm": moe.moe_grouped_gemm, "dgrad": moe.moe_grouped_gemm_dgrad, "wgrad": moe.moe_grouped_gemm_wgrad,
         "orthogonalize": moe.moe_orthogonalize}[name]
    return f(*tensors, **kw)


def operands(name):
    E, rows, N, K = 4, 512, 1024, 1536  # some MB each: blocks that the allocator hands out whole
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * rows
    x, dy = gauss(E * rows, K).bfloat16(), gauss(E * rows, N, seed=1).bfloat16()
    w = (gauss(E, N, K, seed=2) * K ** -0.5).bfloat16()
    return {"gemm": (x, off, w), "dgrad": (dy, off, w), "wgrad": (dy, x, off), "orthogonalize": (gauss(2, 700, 1024, seed=3),)}[name]


@pytest.mark.parametrize("name", CALLS)
def test_operands_let_go_of_after_the_call(cuda_device, name):
    given = operands(name)
    ref, _ = run(name, given)
    shapes = [(t.shape, t.dtype) for t in given if t.is_floating_point()]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)  # some 50 ms
    got, ws = run(name, given, stream=stream)
    del given
    new = [torch.full(s, float("nan"), dtype=d, device="cuda") for s, d in shapes for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(got, ref)
    assert moe.moe_get_device_error(ws) == 0
    assert all(torch.isnan(t).all() for t in new)


def test_a_call_with_stream_can_be_captured(cuda_device):
    x, off, w = operands("gemm")
    ref, ws = moe.moe_grouped_gemm(x, off, w)
    y = torch.zeros_like(ref)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        moe.moe_grouped_gemm(x, off, w, out=y, ws=ws, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
