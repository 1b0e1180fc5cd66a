"""The grouped products and the orthogonalisation on the host (no GPU needed): bad arguments are
refused before anything touches the device.  The pointers are made up, so no call here may pass
validation when a GPU is present."""
import pytest
import torch

import sparse_mixture_experts_16_b200 as moe
from sparse_mixture_experts_16_b200 import build as moe_build

X, OFF, W, OUT, WS = 0x1000, 0x2000, 0x3000, 0x4000, 0x100000


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


def _rows(L, name, **kw):
    a = dict(x=X, off=OFF, w=W, M=100, E=4, N=64, K=72, dtype=0, out_dtype=0, out=OUT, ws=WS,
             ws_bytes=L.moe_grouped_gemm_workspace_size(100))
    a.update(kw)
    return getattr(L, name)(a["x"], a["off"], a["w"], a["M"], a["E"], a["N"], a["K"], a["dtype"], a["out_dtype"],
                            a["out"], a["ws"], a["ws_bytes"], None)


BAD_ROWS = [
    (dict(M=-1), 1), (dict(E=0), 1), (dict(N=0), 1), (dict(K=0), 1),
    (dict(dtype=2, out_dtype=2), 1),       # fp32 operands
    (dict(dtype=3), 1), (dict(out_dtype=1), 1), (dict(dtype=1, out_dtype=0), 1),
    (dict(N=60), 2), (dict(K=12), 2), (dict(E=1025), 2), (dict(N=65544), 2), (dict(K=65544), 2),
    (dict(M=2**31 - 1, N=65536), 2),       # tile numbers past 32 bits
    (dict(x=None), 1), (dict(off=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(x=X + 8), 3), (dict(w=W + 2), 3), (dict(out=OUT + 8), 3), (dict(off=OFF + 2), 3), (dict(ws=WS + 128), 3),
]


@pytest.mark.parametrize("name", ["moe_grouped_gemm", "moe_grouped_gemm_dgrad"])
@pytest.mark.parametrize("kw,status", BAD_ROWS, ids=[str(b[0]) for b in BAD_ROWS])
def test_rows_products_refuse(L, name, kw, status):
    if "M" in kw and kw["M"] > 0:
        kw = dict(kw, ws_bytes=L.moe_grouped_gemm_workspace_size(kw["M"]))
    assert _rows(L, name, **kw) == status


def test_rows_products_refuse_a_small_workspace(L):
    need = L.moe_grouped_gemm_workspace_size(100)
    assert need % 256 == 0
    assert _rows(L, "moe_grouped_gemm", ws_bytes=need - 1) == 4
    assert L.moe_grouped_gemm_workspace_size(-1) == 0
    # one token's workspace is a fraction of a prompt's
    assert L.moe_grouped_gemm_workspace_size(4) < L.moe_grouped_gemm_workspace_size(4096) // 4
    assert L.moe_grouped_gemm_workspace_size(256) == L.moe_grouped_gemm_workspace_size(1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(E=0), 1), (dict(dtype=2), 1), (dict(N=20), 2), (dict(K=20), 2), (dict(E=1025), 2),
    (dict(dy=None), 1), (dict(x=None), 1), (dict(off=None), 1), (dict(dw=None), 1), (dict(ws=None), 1),
    (dict(dy=X + 8), 3), (dict(x=W + 8), 3), (dict(dw=OUT + 4), 3), (dict(ws=WS + 16), 3), (dict(less=1), 4),
])
def test_wgrad_refuses(L, kw, status):
    a = dict(dy=X, x=W, off=OFF, M=100, E=4, N=64, K=72, dtype=0, dw=OUT, ws=WS, less=0)
    a.update(kw)
    need = L.moe_grouped_gemm_wgrad_workspace_size(max(1, a["N"]))
    assert L.moe_grouped_gemm_wgrad(a["dy"], a["x"], a["off"], a["M"], a["E"], a["N"], a["K"], a["dtype"], a["dw"],
                                    a["ws"], need - a["less"], None) == status
    assert L.moe_grouped_gemm_wgrad_workspace_size(0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(M=0), 1), (dict(N=-3), 1), (dict(steps=0), 1), (dict(steps=17), 1), (dict(dtype=1), 1),
    (dict(M=65537), 2), (dict(N=65537), 2), (dict(g=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(g=X + 4), 3), (dict(out=OUT + 2), 3), (dict(ws=WS + 8), 3), (dict(less=1), 4),
])
def test_orthogonalize_refuses(L, kw, status):
    a = dict(g=X, dtype=2, B=3, M=40, N=50, steps=5, out=OUT, ws=WS, less=0)
    a.update(kw)
    need = max(L.moe_orthogonalize_workspace_size(a["B"], a["M"], a["N"]), 256)
    assert L.moe_orthogonalize(a["g"], a["dtype"], a["B"], a["M"], a["N"], a["steps"], a["out"], a["ws"],
                               need - a["less"], None) == status


def test_orthogonalize_workspace(L):
    size = L.moe_orthogonalize_workspace_size
    assert size(0, 4, 4) == size(1, 0, 4) == size(1, 4, 65537) == 0
    assert size(1, 33, 17) % 256 == 0
    # large matrices go through a bounded number at a time
    assert size(512, 2048, 7168) == size(64, 2048, 7168) < 1 << 30
    assert size(1, 2048, 7168) < size(2, 2048, 7168)


@pytest.mark.parametrize("M,E,status", [
    (2**31 - 65535, 1, 2), (2**31 - 1, 8, 2),   # rounding up to tiles would pass 32 bits
    (2**30, 1024, 2),                           # offsets 0, M, 0, M, ... would make 2^31 tiles
    (2**31 - 65536, 1, 3), (2**28 - 256, 1023, 3),  # large enough: the next check, alignment, refuses these
])
def test_products_refuse_rows_past_32_bits(L, M, E, status):
    need = L.moe_grouped_gemm_workspace_size(M)
    for name in ("moe_grouped_gemm", "moe_grouped_gemm_dgrad"):
        assert _rows(L, name, M=M, E=E, N=8, K=8, x=X + 8, ws_bytes=need) == status
    need = L.moe_grouped_gemm_wgrad_workspace_size(8)
    assert L.moe_grouped_gemm_wgrad(X + 8, W, OFF, M, E, 8, 8, 0, OUT, WS, need, None) == status


def test_python_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    w = torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, off, w)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x.float(), off, w.float())
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_dgrad(x[0], off, w)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_wgrad(x, x, off)
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(torch.zeros(4, 4))
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(torch.zeros(4, 4, dtype=torch.float64))


def test_python_finds_the_operands_device_among_keywords():
    class Stream:
        device = torch.device("cuda", 0)

    for kwargs in (dict(steps=5, g=torch.zeros(4, 4)), dict(out=None, g=torch.zeros(4, 4))):
        with pytest.raises(ValueError, match="expected a stream on cpu"):
            moe.moe_orthogonalize(**kwargs, stream=Stream())


def test_python_refuses_sizes_past_32_bits():
    big = 2 ** 32 + 8  # its lower 32 bits would be a valid size
    rows = torch.zeros(1, 8, dtype=torch.bfloat16).expand(big, 8)
    w = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: moe.moe_grouped_gemm(rows, off, w), lambda: moe.moe_grouped_gemm_dgrad(rows, off, w),
                 lambda: moe.moe_grouped_gemm_wgrad(rows, rows, off),
                 lambda: moe.moe_orthogonalize(torch.zeros(1, 1, 1).expand(big, 1, 1)),
                 lambda: moe.moe_orthogonalize(torch.zeros(1, 1).expand(2, big))):
        with pytest.raises(moe.MoeError, match="UNSUPPORTED_SHAPE"):
            call()
