"""Results that stay fp32 are drained every 512 terms and added with rounding.  Lengths at which a sum without
drains is far outside the limit: of all-positive terms it loses about 4e-9 to 5e-9 of itself per term (measured on a
library product with fp32 results: 2.2e-6 at 1024, 1.4e-5 at 4096, 8.2e-5 at 16384), of terms of random
signs a quarter of that."""
import pytest
import torch

import sparse_mixture_experts_16_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("length", [4096, 8192, 16384, 65536])
def test_drained_sums(cuda_device, length, dtype):
    """In a piece of 512 terms each product, and in each of the 32 instructions the sum so far, is aligned to the
    largest addend and loses less than a step of 24 bits, 2^-23 of that: of what the piece has come to, half of the
    piece on average as all terms are positive.  So a piece loses at most (512 + 32) / 2 x 2^-23 of itself: the 22-bit
    products of fp16 come near one in ten of that, the 16-bit ones of bf16 lose less.  Adding a piece rounds at
    most 2^-24 of the sum so far, half of all on average.  (Without drains 16384 terms would be 8e-5 off, 65536 3e-4.)"""
    limit = (512 + 32) / 2 * 2.0 ** -23 + length / 512 / 2 * 2.0 ** -24 + 2.0 ** -24
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn(length, 128, generator=gen, device="cuda").abs().to(dtype) for _ in range(2))
    ref = dy.double().T @ x.double()
    off = torch.tensor([0, length], dtype=torch.int32, device="cuda")
    dw, _ = moe.moe_grouped_gemm_wgrad(dy, x, off)
    assert float((dw[0].double() - ref).norm() / ref.norm()) < limit
    rows = torch.tensor([0, 128], dtype=torch.int32, device="cuda")
    y, _ = moe.moe_grouped_gemm(dy.T.contiguous(), rows, x.T.contiguous()[None], out_dtype=torch.float32)
    assert float((y.double() - ref).norm() / ref.norm()) < limit
    dx, _ = moe.moe_grouped_gemm_dgrad(dy.T.contiguous(), rows, x[None], out_dtype=torch.float32)
    assert float((dx.double() - ref).norm() / ref.norm()) < limit
