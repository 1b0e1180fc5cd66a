"""What moe_orthogonalize's workspace holds (host only): the matrices that run side by side, not the batch."""
import pytest

import sparse_mixture_experts_16_b200 as moe
from sparse_mixture_experts_16_b200 import build as moe_build


@pytest.fixture(scope="module")
def size():
    moe_build.build()
    return moe.lib().moe_orthogonalize_workspace_size


@pytest.mark.parametrize("M,N", [(1, 65536), (8, 65536), (64, 65536), (64, 7168), (7168, 64), (32, 6645), (43, 659), (1, 1)])
@pytest.mark.parametrize("B", [1, 64, 256, 592, 100000])
def test_short_sides_need_at_most_90_mb(size, B, M, N):
    """64 MB of fp32 between rounds of five steps, Gram matrices and products of 592 blocks"""
    assert 0 < size(B, M, N) <= 90e6


@pytest.mark.parametrize("B,M,N", [(18, 24326, 7681), (512, 2048, 7168), (300, 128, 128), (1, 65536, 65536), (7, 65536, 65),
                                   (592, 65, 65536)])
def test_other_sides_need_a_bounded_number_of_matrices(size, B, M, N):
    one = 6 * M * ((N + 15) // 16 * 16) + 4 * min(M, N) * ((min(M, N) + 15) // 16 * 16)
    assert 0 < size(B, M, N) <= max(1.4e9, one + 40e6)
